// fs_fp8_stream_scores.hip -- streaming kernels of the 8-bit head that score tokens.
#include "fs_fp8_stream.hpp"

namespace fs {

hipError_t stream_scores(Fp8Args& a, hipStream_t stream) { return launch_fp8_rows<kTokenScores>(a, stream); }

}  // namespace fs
