// fs_fp8_tile_samples.hip -- block-tiled kernels of the 8-bit head that sample.
#include "fs_fp8_tile.hpp"

namespace fs {

// By exact products: a row of W along h loses 8e-6 of its logit to the 8-bit instructions'
// cut, which at T = 0.3 is 2e-3 of a logit of 82, twice what a winning score may be off.
// They cost nothing while memory bounds the call (64 rows on 128256 x 4096: 110 us, 107 by
// the rounded ones), half or more beyond (256 rows 231 and 163, 1024 850 and 565).
hipError_t tile_samples(Fp8Args& a, hipStream_t stream) {
  return launch_fp8_tiles<kSamples, true>(a, stream);
}

}  // namespace fs
