// fs_fp8_stream_samples.hip -- streaming kernels of the 8-bit head that sample.
#include "fs_fp8_stream.hpp"

namespace fs {

hipError_t stream_samples(Fp8Args& a, hipStream_t stream) { return launch_fp8_rows<kSamples>(a, stream); }

}  // namespace fs
