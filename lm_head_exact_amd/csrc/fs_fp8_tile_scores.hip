// fs_fp8_tile_scores.hip -- block-tiled kernels of the 8-bit head that score tokens.
#include "fs_fp8_tile.hpp"

namespace fs {

// A log-sum-exp of few entries (and of few that count, where T is small) does not average
// the 8-bit instructions' rounding out: with temperatures from 0.3, log-probabilities on
// 700 to 2000 entries are 1.2e-6 of their norm off, exact products 8e-8; on 20000 6e-7 to
// 9e-7, and where all T are 1 at most 3e-7 from 700 on.  Exact products cost small calls
// nothing (1656 rows of 512 on 1977 20.6 us) and large ones up to half (8000 rows of 2048
// on 4000 90 and 132; 2427 of 896 on 41419 116 and 177).  They cost up to 64 rows next to
// nothing on any vocabulary, whose reading bounds the call: 64 on 128256 x 4096 107 us, 104
// by the rounded ones, on 16032 x 8192 38 and 34; 65 rows 132 and 105, 256 218 and 143.
constexpr int32_t kFewEntries = 8192, kFewRows = 64;

hipError_t tile_scores(Fp8Args& a, hipStream_t stream) {
  return a.V <= kFewEntries || a.B <= kFewRows ? launch_fp8_tiles<kTokenScores, true>(a, stream)
                                               : launch_fp8_tiles<kTokenScores>(a, stream);
}

}  // namespace fs
