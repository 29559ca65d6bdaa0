// fs_fp8_tile_samples.hip -- block-tiled kernels of the 8-bit head that sample.
#include "fs_fp8_tile.hpp"

namespace fs {

hipError_t tile_samples(Fp8Args& a, hipStream_t stream) { return launch_fp8_tiles<kSamples>(a, stream); }

}  // namespace fs
