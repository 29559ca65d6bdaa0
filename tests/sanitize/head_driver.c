/* Drives the host paths of the cross entropy and of the 8-bit head (argument checks,
 * size arithmetic, tile rules, the fault-injection hook): invalid arguments, extreme
 * sizes and, under FS_FAULT_INJECT=launch, valid ones.  Nothing is launched and no
 * pointer is touched on the device. */
#define _POSIX_C_SOURCE 200809L
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "flashsample.h"

static int failures = 0;
#define EXPECT(cond)                                                      \
  do {                                                                    \
    if (!(cond)) {                                                        \
      fprintf(stderr, "line %d: %s (%s)\n", __LINE__, #cond, fs_last_error()); \
      ++failures;                                                         \
    }                                                                     \
  } while (0)

#define P ((void*)(uintptr_t)0x10000)
#define F ((float*)(uintptr_t)0x10000)
#define I ((int32_t*)(uintptr_t)0x10000)
#define WS ((void*)(uintptr_t)0x20000)
#define BIG ((size_t)1 << 62)

static void cross_entropy(fs_status valid) {
  const int32_t Bs[] = {0, 1, 17, 300, 16500, 1 << 22}, Ds[] = {8, 40, 4096, 1 << 20};
  const int32_t Vs[] = {1, 15, 1000, 128256, 300000, 2147483135};
  for (size_t b = 0; b < sizeof Bs / sizeof *Bs; ++b)
    for (size_t d = 0; d < sizeof Ds / sizeof *Ds; ++d)
      for (size_t v = 0; v < sizeof Vs / sizeof *Vs; ++v)
        for (int32_t grads = 0; grads < 2; ++grads) {
          const int32_t B = Bs[b], D = Ds[d], V = Vs[v];
          void* g = grads ? P : NULL;
          const size_t need = fs_cross_entropy_workspace_bytes(B, D, V, grads);
          EXPECT(need > 0 && need % 256 == 0);
          fs_status s = fs_cross_entropy(P, P, B, D, V, I, 0.1, 1e-4, 1, 1.0, F, F, g, g, WS, BIG, NULL);
          EXPECT(s == valid || s == FS_ERR_UNSUPPORTED);
          EXPECT(fs_cross_entropy(P, P, B, D, V, I, 0.0, 0.0, 0, -2.0, F, F, g, g, WS, need - 1, NULL) ==
                 FS_ERR_WORKSPACE);
        }
  EXPECT(fs_cross_entropy_workspace_bytes(1, 8, 2147483647, 1) == 0);
  EXPECT(fs_cross_entropy(P, P, 1, 8, 1, I, NAN, 0.0, 1, 1.0, F, F, P, P, WS, BIG, NULL) == FS_ERR_INVALID_ARG);
  EXPECT(fs_cross_entropy(P, P, 1, 8, 1, I, 0.0, INFINITY, 1, 1.0, F, F, P, P, WS, BIG, NULL) ==
         FS_ERR_INVALID_ARG);
  EXPECT(fs_cross_entropy(P, P, -2147483647 - 1, 8, 1, I, 0.0, 0.0, 1, 1.0, F, F, P, P, WS, BIG, NULL) ==
         FS_ERR_INVALID_ARG);
}

static void eight_bit(fs_status valid) {
  const int32_t Bs[] = {0, 1, 16, 17, 33, 777, 1 << 22}, Ds[] = {64, 4096, 5184, 8192, 16384};
  const int32_t Vs[] = {1, 15, 1000, 128256, 2147483135};
  for (size_t b = 0; b < sizeof Bs / sizeof *Bs; ++b)
    for (size_t d = 0; d < sizeof Ds / sizeof *Ds; ++d)
      for (size_t v = 0; v < sizeof Vs / sizeof *Vs; ++v) {
        const int32_t B = Bs[b], D = Ds[d], V = Vs[v];
        const fs_status want = B == 0 ? FS_OK : valid;
        const size_t need = fs_fp8_workspace_bytes(B, D, V);
        EXPECT(need > 0);
        fs_status s = fs_logits_fp8(P, P, P, B, D, V, 1, P, V, WS, BIG, NULL);
        EXPECT(s == want || s == FS_ERR_UNSUPPORTED);
        s = fs_token_logprobs_fp8(P, P, P, B, D, V, 0, NULL, I, F, F, WS, BIG, NULL);
        EXPECT(s == want || s == FS_ERR_UNSUPPORTED);
        s = fs_sample_fp8(P, P, P, B, D, V, 0, F, 1, 2, I, F, WS, BIG, NULL);
        EXPECT(s == want || s == FS_ERR_UNSUPPORTED);
        if (B > 0 && s != FS_ERR_UNSUPPORTED)
          EXPECT(fs_sample_fp8(P, P, P, B, D, V, 0, F, 1, 2, I, F, WS, need - 1, NULL) == FS_ERR_WORKSPACE);
        const size_t bytes = fs_fp8_weights_bytes(V, D, 1);
        EXPECT(bytes >= (size_t)V * D && bytes % 1024 == 0);
        s = fs_quantize_weights_fp8(P, V, D, 1, P, bytes, P, NULL);
        EXPECT(s == valid || s == FS_ERR_UNSUPPORTED);
        EXPECT(fs_quantize_weights_fp8(P, V, D, 0, P, (size_t)V * D - 1, P, NULL) == FS_ERR_WORKSPACE);
        EXPECT(fs_pack_weights_fp8(P, V, D, P, bytes, NULL) == valid);
      }
  EXPECT(fs_logits_fp8(P, P, P, 2, 64, 10, 1, P, INT64_MAX, WS, BIG, NULL) == FS_ERR_INVALID_ARG);
  EXPECT(fs_logits_fp8(P, P, P, 2, 64, 10, 1, P, INT64_MIN, WS, BIG, NULL) == FS_ERR_INVALID_ARG);
  EXPECT(fs_sample_fp8(P, P, P, 2, 64, 10, 2147483640, F, 1, 2, I, F, WS, BIG, NULL) == FS_ERR_INVALID_ARG);
  EXPECT(fs_fp8_weights_bytes(-1, 64, 1) == 0 && fs_fp8_workspace_bytes(1, 65, 1) == 0);
}

int main(void) {
  setenv("FS_FAULT_INJECT", "launch", 1);
  cross_entropy(FS_ERR_HIP);
  eight_bit(FS_ERR_HIP);
  if (failures) return 1;
  printf("all head host paths ran clean\n");
  return 0;
}
