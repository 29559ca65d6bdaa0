// fs_fp8.hip -- entry points of the LM head in 8-bit floating point.
#include "fs_fp8.hpp"

#include <algorithm>

#include "fs_host.hpp"
#include "fs_internal.hpp"

namespace fs {

namespace {

struct Fp8Layout {
  int32_t Dp, Bp;
  size_t hq, hscale, part, target, total;
  Fp8Layout(int32_t B, int32_t D, int32_t V) {
    const bool streams = fp8_streams(B, D);
    Dp = static_cast<int32_t>(round_up(D, kQuantBlock));
    Bp = static_cast<int32_t>(round_up(B, 256));
    // (a streaming block takes a group of 16 rows at least)
    const size_t S = streams ? std::min(kMaxFp8StreamBlocks, fp8_groups(V))
                             : (static_cast<size_t>(V) + rows_of(fp8_tile(B, D, V)) - 1) /
                                   rows_of(fp8_tile(B, D, V));
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t o = at;
      at += round_up(bytes, 256);
      return o;
    };
    hq = take(streams ? 0 : static_cast<size_t>(B) * Dp);
    hscale = take(streams ? 0 : static_cast<size_t>(quant_blocks(D)) * Bp);
    part = take(8 * S * B);
    target = take(4ull * B);
    total = at;
  }
};

bool fp8_sizes_ok(int32_t B, int32_t D, int32_t V) {
  return B >= 0 && D >= 64 && D % 64 == 0 && V >= 1 && B <= kMaxFp8B && D <= kMaxFp8D &&
         V <= kMaxVocab;
}

fs_status check_head(const char* who, int32_t D, int32_t V, int32_t multiple) {
  if (D < multiple || D % multiple != 0)
    return fail(FS_ERR_INVALID_ARG, "%s: D must be a positive multiple of %d (got %d)", who, multiple,
                D);
  if (V < 1) return fail(FS_ERR_INVALID_ARG, "%s: V must be >= 1 (got %d)", who, V);
  if (D > kMaxFp8D || V > kMaxVocab)
    return fail(FS_ERR_UNSUPPORTED, "%s: D=%d, V=%d exceed the %d elements or %d entries a call can "
                "take", who, D, V, kMaxFp8D, kMaxVocab);
  return FS_OK;
}

// Checks what the three products share and fills the arguments.
fs_status prepare(const char* who, const void* h, const void* W, const void* scale, int32_t B,
                  int32_t D, int32_t V, int32_t vocab_offset, void* workspace,
                  size_t workspace_bytes, Fp8Args& a) {
  if (B < 0) return fail(FS_ERR_INVALID_ARG, "%s: B must be >= 0 (got %d)", who, B);
  const fs_status st = check_head(who, D, V, 64);
  if (st != FS_OK) return st;
  if (vocab_offset < 0 || static_cast<int64_t>(vocab_offset) + V > 2147483647)
    return fail(FS_ERR_INVALID_ARG, "%s: vocab_offset and vocab_offset + V must be in [0, 2^31 - 1]"
                " (got %d, V = %d)", who, vocab_offset, V);
  if (B > kMaxFp8B)
    return fail(FS_ERR_UNSUPPORTED, "%s: B=%d exceeds the %d rows a call can take", who, B, kMaxFp8B);
  if (!fp8_streams(B, D) && B > 0) {  // (streaming grids are bounded by the device)
    const LogitsTile t = fp8_tile(B, D, V);
    const int64_t tiles = (static_cast<int64_t>(V) + rows_of(t) - 1) / rows_of(t) *
                          ((B + tokens_of(t) - 1) / tokens_of(t));
    if (!grid_fits(tiles + 7, threads_of(t)) ||
        !grid_fits(B, static_cast<int64_t>(round_up(round_up(D, kQuantBlock) / 16, 64))))
      return fail(FS_ERR_UNSUPPORTED, "%s: B=%d, D=%d, V=%d exceed the launch grid", who, B, D, V);
  }
  if (B == 0) return FS_OK;
  if (!h || !W || !scale || !workspace)
    return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (!aligned(h, 16) || !aligned(W, 16))
    return fail(FS_ERR_INVALID_ARG, "%s: h and W must be 16-byte aligned", who);
  if (!aligned(workspace, 256))
    return fail(FS_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  const Fp8Layout lay(B, D, V);
  if (workspace_bytes < lay.total)
    return fail(FS_ERR_WORKSPACE, "%s: workspace of %zu bytes is below the %zu required", who,
                workspace_bytes, lay.total);
  char* ws = static_cast<char*>(workspace);
  a = Fp8Args{};
  a.w = static_cast<const uint8_t*>(W);
  a.wscale = static_cast<const uint8_t*>(scale);
  a.h = static_cast<const __bf16*>(h);
  a.B = B;
  a.D = D;
  a.V = V;
  a.KB = quant_blocks(D);
  a.vocab_offset = vocab_offset;
  a.hq = reinterpret_cast<uint8_t*>(ws + lay.hq);
  a.hscale = reinterpret_cast<uint8_t*>(ws + lay.hscale);
  a.Dp = lay.Dp;
  a.Bp = lay.Bp;
  a.part = reinterpret_cast<float2*>(ws + lay.part);
  a.target = reinterpret_cast<float*>(ws + lay.target);
  return FS_OK;
}

using Launch = hipError_t (*)(Fp8Args&, hipStream_t);

hipError_t launch_product(Fp8Args& a, Launch stream_kernels, Launch tiles, hipStream_t s) {
  if (fp8_streams(a.B, a.D)) return stream_kernels(a, s);
  const hipError_t e = launch_quantize_rows(a, s);
  return e == hipSuccess ? tiles(a, s) : e;
}

}  // namespace
}  // namespace fs

extern "C" {

FS_API size_t fs_fp8_weights_bytes(int32_t V, int32_t D, int32_t packed) {
  using namespace fs;
  if (V < 1 || D < 8 || D % (packed ? 64 : 8) != 0 || D > kMaxFp8D || V > kMaxVocab) return 0;
  return (packed ? 16 * static_cast<size_t>(fp8_groups(V)) : static_cast<size_t>(V)) * D;
}

FS_API fs_status fs_quantize_weights_fp8(const void* W, int32_t V, int32_t D, int32_t packed,
                                         void* out_q, size_t q_bytes, void* out_scale,
                                         void* stream) {
  using namespace fs;
  const char* who = "fs_quantize_weights_fp8";
  const fs_status st = check_head(who, D, V, packed ? 64 : 8);
  if (st != FS_OK) return st;
  if (!W || !out_q || !out_scale) return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (!aligned(W, 16) || !aligned(out_q, 16))
    return fail(FS_ERR_INVALID_ARG, "%s: W and the quantised weights must be 16-byte aligned", who);
  const size_t need = fs_fp8_weights_bytes(V, D, packed);
  if (q_bytes < need)
    return fail(FS_ERR_WORKSPACE, "%s: buffer of %zu bytes is below the %zu required", who, q_bytes,
                need);
  if (!grid_fits(static_cast<int64_t>(quant_blocks(V)) * ((quant_blocks(D) + 3) / 4), 1024))
    return fail(FS_ERR_UNSUPPORTED, "%s: D=%d, V=%d exceed the launch grid", who, D, V);
  if (start_launches()) return injected_failure(who);
  const hipError_t e = launch_quantize_weights(
      static_cast<const __bf16*>(W), V, D, packed != 0, static_cast<uint8_t*>(out_q),
      static_cast<uint8_t*>(out_scale), static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FS_OK : hip_fail(e, "quantising launch");
}

FS_API fs_status fs_pack_weights_fp8(const void* q, int32_t V, int32_t D, void* out_packed,
                                     size_t packed_bytes, void* stream) {
  using namespace fs;
  const char* who = "fs_pack_weights_fp8";
  const fs_status st = check_head(who, D, V, 64);
  if (st != FS_OK) return st;
  if (!q || !out_packed) return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (!aligned(q, 16) || !aligned(out_packed, 16))
    return fail(FS_ERR_INVALID_ARG, "%s: both buffers must be 16-byte aligned", who);
  const size_t need = fs_fp8_weights_bytes(V, D, 1);
  if (packed_bytes < need)
    return fail(FS_ERR_WORKSPACE, "%s: buffer of %zu bytes is below the %zu required", who,
                packed_bytes, need);
  if (start_launches()) return injected_failure(who);
  const hipError_t e = launch_pack_fp8(static_cast<const uint8_t*>(q), V, D,
                                       static_cast<uint8_t*>(out_packed),
                                       static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FS_OK : hip_fail(e, "packing launch");
}

FS_API size_t fs_fp8_workspace_bytes(int32_t B, int32_t D, int32_t V) {
  return fs::fp8_sizes_ok(B, D, V) ? fs::Fp8Layout(B > 0 ? B : 1, D, V).total : 0;
}

FS_API fs_status fs_logits_fp8(const void* h, const void* W_packed, const void* W_scale, int32_t B,
                               int32_t D, int32_t V, int32_t out_fp32, void* out_logits,
                               int64_t row_pitch, void* workspace, size_t workspace_bytes,
                               void* stream) {
  using namespace fs;
  const char* who = "fs_logits_fp8";
  Fp8Args a;
  const fs_status st =
      prepare(who, h, W_packed, W_scale, B, D, V, 0, workspace, workspace_bytes, a);
  if (st != FS_OK) return st;
  if (row_pitch < V || row_pitch > (int64_t{1} << 40))
    return fail(FS_ERR_INVALID_ARG, "%s: row_pitch must be in [V, 2^40] (got %lld)", who,
                static_cast<long long>(row_pitch));
  if (B == 0) return FS_OK;
  const size_t size = out_fp32 ? 4 : 2;
  if (!out_logits) return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (!aligned(out_logits, size))
    return fail(FS_ERR_INVALID_ARG, "%s: the logits must be aligned to their size", who);
  if (start_launches()) return injected_failure(who);
  a.out = out_logits;
  a.ld = row_pitch;
  a.lines = aligned(out_logits, 128) && row_pitch * size % 128 == 0;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = out_fp32 ? launch_product(a, stream_logits_f32, tile_logits_f32, s)
                                : launch_product(a, stream_logits_bf16, tile_logits_bf16, s);
  return e == hipSuccess ? FS_OK : hip_fail(e, "8-bit logits launch");
}

FS_API fs_status fs_token_logprobs_fp8(const void* h, const void* W_packed, const void* W_scale,
                                       int32_t B, int32_t D, int32_t V, int32_t vocab_offset,
                                       const float* temperature, const int32_t* token_ids,
                                       float* out_logprob, float* out_lse, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  using namespace fs;
  const char* who = "fs_token_logprobs_fp8";
  Fp8Args a;
  const fs_status st =
      prepare(who, h, W_packed, W_scale, B, D, V, vocab_offset, workspace, workspace_bytes, a);
  if (st != FS_OK || B == 0) return st;
  if (!token_ids || !out_logprob || !out_lse)
    return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (!aligned(token_ids, 4) || !aligned(out_logprob, 4) || !aligned(out_lse, 4) ||
      !aligned(temperature, 4))
    return fail(FS_ERR_INVALID_ARG, "%s: per-row arrays must be 4-byte aligned", who);
  if (start_launches()) return injected_failure(who);
  a.temperature = temperature;
  a.ids = token_ids;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = launch_product(a, stream_scores, tile_scores, s);
  if (e != hipSuccess) return hip_fail(e, "8-bit log-probability launch");
  ScoreArgs c{};
  c.B = B;
  c.D = D;
  c.V = V;
  c.vocab_offset = vocab_offset;
  c.temperature = temperature;
  c.ids = token_ids;
  c.part = a.part;
  c.target = a.target;
  c.S = a.S;
  e = launch_score_close(c, out_logprob, out_lse, s);
  return e == hipSuccess ? FS_OK : hip_fail(e, "log-probability merge launch");
}

FS_API fs_status fs_sample_fp8(const void* h, const void* W_packed, const void* W_scale, int32_t B,
                               int32_t D, int32_t V, int32_t vocab_offset,
                               const float* temperature, uint64_t seed, uint64_t step,
                               int32_t* out_ids, float* out_maxval, void* workspace,
                               size_t workspace_bytes, void* stream) {
  using namespace fs;
  const char* who = "fs_sample_fp8";
  Fp8Args a;
  const fs_status st =
      prepare(who, h, W_packed, W_scale, B, D, V, vocab_offset, workspace, workspace_bytes, a);
  if (st != FS_OK) return st;
  if (vocab_offset % 4 != 0)
    return fail(FS_ERR_INVALID_ARG, "%s: vocab_offset must be a multiple of 4 (got %d)", who,
                vocab_offset);
  if (B == 0) return FS_OK;
  if (!temperature || !out_ids || !out_maxval)
    return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (!aligned(temperature, 4) || !aligned(out_ids, 4) || !aligned(out_maxval, 4))
    return fail(FS_ERR_INVALID_ARG, "%s: per-row arrays must be 4-byte aligned", who);
  if (start_launches()) return injected_failure(who);
  const Fp8Layout lay(B, D, V);
  a.temperature = temperature;
  a.seed = seed;
  a.step = step;
  a.part_val = reinterpret_cast<float*>(a.part);
  // (the launchers set S: the ids follow the most values there can be)
  const size_t most = (lay.target - lay.part) / 8;
  a.part_idx = reinterpret_cast<int32_t*>(a.part_val + most);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = launch_product(a, stream_samples, tile_samples, s);
  if (e != hipSuccess) return hip_fail(e, "8-bit sampler launch");
  e = launch_merge(a.part_val, a.part_idx, a.S, B, 1, a.S, out_ids, out_maxval, s);
  return e == hipSuccess ? FS_OK : hip_fail(e, "merge launch");
}

}  // extern "C"
