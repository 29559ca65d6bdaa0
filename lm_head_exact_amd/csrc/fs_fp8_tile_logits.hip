// fs_fp8_tile_logits.hip -- block-tiled kernels of the 8-bit head that write logits.
#include "fs_fp8_tile.hpp"

namespace fs {

hipError_t tile_logits_bf16(Fp8Args& a, hipStream_t stream) {
  return launch_fp8_tiles<kLogitsBf16>(a, stream);
}
hipError_t tile_logits_f32(Fp8Args& a, hipStream_t stream) {
  return launch_fp8_tiles<kLogitsF32>(a, stream);
}

}  // namespace fs
