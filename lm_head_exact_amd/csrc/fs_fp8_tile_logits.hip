// fs_fp8_tile_logits.hip -- block-tiled kernels of the 8-bit head that write logits.
#include "fs_fp8_tile.hpp"

namespace fs {

// bf16 logits take the 8-bit instructions: what these cut (1e-5 of a logit, 1.5e-5 of the
// logits' spread) is far below the result's own rounding.  Logits in fp32 are sums of exact
// products (64 rows on 128256 x 4096 104 us, 103 by the rounded ones; 256 rows 223 and 154,
// 1024 814 and 547).
hipError_t tile_logits_bf16(Fp8Args& a, hipStream_t stream) {
  return launch_fp8_tiles<kLogitsBf16>(a, stream);
}
hipError_t tile_logits_f32(Fp8Args& a, hipStream_t stream) {
  return launch_fp8_tiles<kLogitsF32, true>(a, stream);
}

}  // namespace fs
