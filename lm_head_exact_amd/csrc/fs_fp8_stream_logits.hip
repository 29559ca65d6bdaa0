// fs_fp8_stream_logits.hip -- streaming kernels of the 8-bit head that write logits.
#include "fs_fp8_stream.hpp"

namespace fs {

hipError_t stream_logits_bf16(Fp8Args& a, hipStream_t stream) {
  return launch_fp8_rows<kLogitsBf16>(a, stream);
}
hipError_t stream_logits_f32(Fp8Args& a, hipStream_t stream) {
  return launch_fp8_rows<kLogitsF32>(a, stream);
}

}  // namespace fs
