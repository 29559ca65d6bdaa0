// fs_fp8_tile_scores.hip -- block-tiled kernels of the 8-bit head that score tokens.
#include "fs_fp8_tile.hpp"

namespace fs {

hipError_t tile_scores(Fp8Args& a, hipStream_t stream) { return launch_fp8_tiles<kTokenScores>(a, stream); }

}  // namespace fs
