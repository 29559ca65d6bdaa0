/* Drives the training operators' host paths (argument checks, size arithmetic,
 * table building, the fault-injection hook): invalid arguments, extreme sizes
 * and, under FS_FAULT_INJECT=launch, valid ones.  Nothing is launched and no
 * pointer is touched on the device. */
#define _POSIX_C_SOURCE 200809L
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

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
#define M ((uint8_t*)(uintptr_t)0x10000)
#define WS ((void*)(uintptr_t)0x20000)
#define BIG ((size_t)1 << 62)

static void logprobs(fs_status valid) {
  const int32_t Bs[] = {0, 1, 16, 17, 33, 300, 1 << 24}, Ds[] = {8, 40, 256, 4096, 8192, 1 << 20};
  const int32_t Vs[] = {1, 15, 1000, 128256, 2147483135};
  for (size_t b = 0; b < sizeof Bs / sizeof *Bs; ++b)
    for (size_t d = 0; d < sizeof Ds / sizeof *Ds; ++d)
      for (size_t v = 0; v < sizeof Vs / sizeof *Vs; ++v) {
        const int32_t B = Bs[b], D = Ds[d], V = Vs[v];
        const size_t need = fs_token_logprobs_workspace_bytes(B, D, V);
        fs_status s = fs_token_logprobs(P, P, B, D, V, 0, F, I, F, F, WS, BIG, NULL);
        EXPECT(s == (B == 0 ? FS_OK : valid) || s == FS_ERR_UNSUPPORTED);
        if (B > 0 && s != FS_ERR_UNSUPPORTED)
          EXPECT(fs_token_logprobs(P, P, B, D, V, 0, NULL, I, F, F, WS, need - 1, NULL) ==
                 FS_ERR_WORKSPACE);
        s = fs_token_logprobs_packed(P, P, B, D, V, 0, F, I, F, F, WS, BIG, NULL);
        EXPECT(s == (D % 32 ? FS_ERR_INVALID_ARG : B == 0 ? FS_OK : valid) || s == FS_ERR_UNSUPPORTED);
        const size_t back = fs_token_logprobs_backward_workspace_bytes(B, D, V);
        EXPECT((back == 0) == (B > (1 << 22)));
        s = fs_token_logprobs_backward(P, P, B, D, V, 0, F, I, F, F, F, P, P, WS, BIG, NULL);
        EXPECT(s == valid || s == FS_ERR_UNSUPPORTED);
      }
  EXPECT(fs_token_logprobs_workspace_bytes(1, 8, 2147483647) == 0);
  EXPECT(fs_token_logprobs_backward_workspace_bytes(1, 8, 2147483647) == 0);
  EXPECT(fs_token_logprobs(P, P, 1, 8, 2147483647, 0, F, I, F, F, WS, BIG, NULL) == FS_ERR_UNSUPPORTED);
  EXPECT(fs_token_logprobs(NULL, P, 1, 8, 1, 0, F, I, F, F, WS, BIG, NULL) == FS_ERR_INVALID_ARG);
  EXPECT(fs_token_logprobs_backward(P, P, 1, 8, 1, 0, F, I, F, F, F, NULL, NULL, WS, BIG, NULL) ==
         FS_ERR_INVALID_ARG);
}

static void losses(fs_status valid) {
  const int32_t Ss[] = {0, 1, 2, 511, 512, 1 << 20}, Ts[] = {0, 1, 4096, 4097, 1 << 24, 2147483647};
  for (size_t a = 0; a < sizeof Ss / sizeof *Ss; ++a)
    for (size_t b = 0; b < sizeof Ts / sizeof *Ts; ++b) {
      const int32_t S = Ss[a], T = Ts[b];
      const size_t need = fs_loss_workspace_bytes(S, T);
      EXPECT(fs_policy_loss(F, F, F, F, M, I, S, T, 1, 0.2, 0.2, 3.0, 0.1, FS_KL_K3, FS_TOKEN_MEAN,
                            1.0, 0, F, F, WS, need, NULL) == valid);
      if (S % 2 == 0)
        EXPECT(fs_preference_loss(F, F, M, I, S / 2, T, FS_PREFERENCE_SIGMOID, 0.1, 0.0, 0.1, 1, 1.0,
                                  1, F, F, F, WS, need, NULL) == valid);
      if (need > 0)
        EXPECT(fs_policy_loss(F, F, NULL, F, NULL, I, S, T, 0, 0.2, 0.2, 0.0, 0.0, FS_KL_K1,
                              FS_SEQUENCE_MEAN, 1.0, 0, F, F, WS, need - 1, NULL) == FS_ERR_WORKSPACE);
    }
  EXPECT(fs_policy_loss(F, F, F, F, M, I, 4, 9000, 0, NAN, 0.2, 0.0, 0.1, FS_KL_K3, FS_TOKEN_MEAN, 1.0,
                        0, F, F, WS, BIG, NULL) == FS_ERR_INVALID_ARG);
  EXPECT(fs_preference_loss(F, F, M, I, 4, 9000, FS_PREFERENCE_IPO, 0.1, 1.0, 0.0, 0, 1.0, 0, F, F, F,
                            WS, BIG, NULL) == FS_ERR_INVALID_ARG);
}

static void clipping(fs_status valid) {
  enum { N = 1000 };
  const void* grads[N];
  void* out[N];
  int64_t numel[N];
  fs_dtype types[N];
  for (int i = 0; i < N; ++i) {
    grads[i] = P;
    out[i] = WS;
    numel[i] = (int64_t)i * 4097 % 100003;
    types[i] = (fs_dtype)(i % 3);
  }
  const int counts[] = {0, 1, 95, 96, 97, N};
  for (size_t c = 0; c < sizeof counts / sizeof *counts; ++c) {
    const int n = counts[c];
    const size_t need = fs_clip_grad_norm_workspace_bytes(numel, n);
    EXPECT(need > 0);
    EXPECT(fs_clip_grad_norm(grads, NULL, numel, types, n, 1.0f, F, WS, need, NULL) == valid);
    EXPECT(fs_clip_grad_norm(grads, out, numel, types, n, INFINITY, F, WS, need, NULL) == valid);
    EXPECT(fs_clip_grad_norm(grads, out, numel, types, n, 1.0f, F, WS, need - 1, NULL) ==
           FS_ERR_WORKSPACE);
  }
  numel[3] = INT64_MAX;
  EXPECT(fs_clip_grad_norm_workspace_bytes(numel, N) == 0);
  EXPECT(fs_clip_grad_norm(grads, NULL, numel, types, N, 1.0f, F, WS, BIG, NULL) == FS_ERR_UNSUPPORTED);
  numel[3] = -1;
  EXPECT(fs_clip_grad_norm(grads, NULL, numel, types, N, 1.0f, F, WS, BIG, NULL) == FS_ERR_INVALID_ARG);
}

int main(void) {
  setenv("FS_FAULT_INJECT", "launch", 1);
  logprobs(FS_ERR_HIP);
  losses(FS_ERR_HIP);
  clipping(FS_ERR_HIP);
  if (failures) return 1;
  printf("all training host paths ran clean\n");
  return 0;
}
