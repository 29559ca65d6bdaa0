// fs_logprob.hip -- log-probabilities of given tokens straight from hidden
// states and the LM head (fs_token_logprobs): the B x V logits stay on chip.
#include <cmath>

#include "fs_host.hpp"
#include "fs_score.hpp"
#include "fs_sampler.hpp"

namespace fs {
namespace {

// ---------------------------------------------------------------------------
// Block-tiled kernel: any B and D.  Grid of vocabulary tiles by token tiles; a
// tile's logits become one pair (maximum, sum of exponentials) per token in
// registers, and the pairs of its waves one in LDS.  1777 tokens on 151936 rows
// of 5120: 2.2 to 2.4 ms, 1.15 to 1.25 PFLOP/s, at 1.8 GHz as the tile loop
// runs there (a bf16 library product of that size: 1.4 PFLOP/s, without
// the reduction and with 540 MB of logits written).
// ---------------------------------------------------------------------------
template <class T>
__global__ __launch_bounds__(T::kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void score_tile_kernel(ScoreArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn_smem[];
  int tile, btile;
  if (!xcd_tile<4>(blockIdx.x, a.S, (a.B + T::TB - 1) / T::TB, tile, btile)) return;
  const int a0 = tile * T::TA, b0 = btile * T::TB;
  f32x4 acc[T::MR][T::NT];
  T::run(a.w, a.h, a0, b0, 0, (a.D + T::BK - 1) / T::BK, acc, dyn_smem);

  const int lane = threadIdx.x & (kWave - 1), li = lane & 15, kb = lane >> 4;
  const int row0 = a0 + T::wave_a() - a.shift, col0 = b0 + T::wave_b();
  float2* red = reinterpret_cast<float2*>(dyn_smem);  // [WA][TB]
  const bool inside = row0 >= 0 && row0 + T::MR * 16 <= a.V;
  static_for<T::NT>([&](auto n) FS_INLINE {
    const int b = col0 + 16 * static_cast<int>(n) + li;
    const int bc = min(b, a.B - 1);
    const float inv_t = score_inv_t(a.temperature, bc);
    const int loc = target_row(a.ids[bc], a.vocab_offset, a.V);
    const bool hit = loc >= row0 && loc < row0 + T::MR * 16;
    const bool plain = inside && __ballot(hit) == 0;
    float m = LseAcc::kMasked, s = 0.0f, zt = 0.0f;
    bool has = false;
    fold_logits<T::MR>([&](auto i) FS_INLINE { return acc[i][n]; }, row0, a.V, loc, plain, inv_t, m,
                       s, zt, has);
    if (has && b < a.B) a.target[b] = zt;
    pair_xor(m, s, 16);
    pair_xor(m, s, 32);
    if (kb == 0) red[(T::wave() / T::WB) * T::TB + T::wave_b() + 16 * n + li] = float2{m, s};
  });
  __syncthreads();
  for (int c = threadIdx.x; c < T::TB; c += T::kThreads) {
    if (b0 + c >= a.B) break;
    float2 p = red[c];
#pragma unroll
    for (int w = 1; w < T::WA; ++w) {
      const float2 o = red[w * T::TB + c];
      pair_merge(p.x, p.y, o.x, o.y);
    }
    a.part[static_cast<size_t>(tile) * a.B + b0 + c] = p;
  }
}

// h with its rows padded by zeros to a multiple of 64 elements.
__global__ __launch_bounds__(256) void pad_rows_kernel(const __bf16* h, int32_t B, int32_t D,
                                                       int32_t Dp, __bf16* out) {
  const int pieces = Dp / 8;
  const int64_t total = static_cast<int64_t>(B) * pieces;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += 256ll * gridDim.x) {
    const int b = static_cast<int>(i / pieces), k = static_cast<int>(i % pieces) * 8;
    const bf16x8 v = k < D ? load_frag(h + static_cast<size_t>(b) * D + k) : zero_frag();
    *reinterpret_cast<bf16x8*>(out + static_cast<size_t>(b) * Dp + k) = v;
  }
}

// ---------------------------------------------------------------------------
// Streaming kernel for up to NT * 16 tokens: bound by reading W once (128256 x
// 4096 in fragment order: one token 148 us, 7.1 TB/s; 32 tokens 158; row-major
// 173, whose 16 rows of a group lie in 16 pages).  A
// block's NW waves split D (KS k-steps of 32 each) and keep their slice of h
// in registers; blocks sweep the 16-row vocabulary groups strided by the
// grid, so that the rows being read form a narrow moving window of W (HBM
// page locality), through a ring of P loads that runs ahead across groups.
// The partial sums meet in LDS; the wave whose turn it is adds them in wave
// order and folds the 16 rows into its running pairs.  k's past D load W's last
// piece again and take zeros of both operands (an infinite entry of that piece
// must not meet a zero of h).
// ---------------------------------------------------------------------------
template <int NT, int NW, int KS, int P, bool PACKED, bool WHOLE>
__global__ __launch_bounds__(NW * kWave) void score_stream_kernel(ScoreArgs a) {
  static_assert(KS % P == 0, "the load ring must tile a group");
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn_smem[];
  f32x4* red = reinterpret_cast<f32x4*>(dyn_smem);  // [2][NW][NT][kWave]
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int li = lane & 15, kb = lane >> 4;
  const int D = a.D, G = gridDim.x;
  const int ngroups = (a.V + a.shift + 15) / 16;
  const int k0 = wave * KS * 32 + 8 * kb;

  bf16x8 hreg[KS][NT];
  float inv_t[NT];
  int loc[NT];
  static_for<NT>([&](auto n) FS_INLINE {
    const int b = n * 16 + li, bc = min(b, a.B - 1);
    const __bf16* hp = a.h.p + static_cast<size_t>(bc) * D;
    static_for<KS>([&](auto s) FS_INLINE {
      const int k = k0 + static_cast<int>(s) * 32;
      hreg[s][n] = load_frag(hp + min(k, D - 8));
      if (k >= D) hreg[s][n] = zero_frag();
    });
    inv_t[n] = score_inv_t(a.temperature, bc);
    loc[n] = b < a.B ? target_row(a.ids[bc], a.vocab_offset, a.V) : -1;
  });
  // The lane's first piece of group t (clamped to the last group), and the
  // piece of its k-step s.  WHOLE: D is 32 * NW * KS, so no step is past D.
  const int last_step = D / 32 - 1;
  auto group = [&](int t) FS_INLINE {
    const int g = min(t, ngroups - 1);
    if constexpr (PACKED)
      return packed_frag(a.w.p, g, D, lane) + (WHOLE ? wave * KS * kPackedStep : 0);
    else
      return a.w.p + static_cast<size_t>(clamp_row(16 * g - a.shift + li, a.V)) * D + (WHOLE ? k0 : 0);
  };
  auto load = [&](const __bf16* p, int s) FS_INLINE {
    if constexpr (PACKED)
      return load_frag<true>(p + (WHOLE ? s : min(wave * KS + s, last_step)) * kPackedStep);
    else
      return load_frag<false>(p + (WHOLE ? 32 * s : min(k0 + 32 * s, D - 8)));
  };
  // The wave's k-steps within D (scalar), and whether the lane's piece of the next
  // one is, where D ends in it.
  const int whole_steps = __builtin_amdgcn_readfirstlane(min(max(D / 32 - wave * KS, 0), KS));
  const bool part = !PACKED && D / 32 >= wave * KS && 8 * kb < D % 32;
  float m[NT], s_[NT];
  static_for<NT>([&](auto n) FS_INLINE {
    m[n] = LseAcc::kMasked;
    s_[n] = 0.0f;
  });
  int g = blockIdx.x;
  const __bf16* wp = group(g);
  const __bf16* wn = group(g + G);
  bf16x8 ring[P];
  static_for<P>([&](auto p) FS_INLINE { ring[p] = load(wp, p); });
  for (int it = 0; g < ngroups; g += G, ++it) {
    f32x4 acc[NT];
    static_for<NT>([&](auto n) FS_INLINE { acc[n] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    // (compared anew for every group: kept, the steps' masks would fill the scalar
    // registers)
    int steps = whole_steps;
    if constexpr (!WHOLE) asm volatile("" : "+s"(steps));
    static_for<KS>([&](auto sc) FS_INLINE {
      constexpr int s = decltype(sc)::value, slot = s % P;
      const bf16x8 w =
          WHOLE || s < steps || (s == steps && part) ? ring[slot] : zero_frag();
      static_for<NT>([&](auto n) FS_INLINE { acc[n] = mfma16(w, hreg[s][n], acc[n]); });
      if constexpr (s + P < KS) ring[slot] = load(wp, s + P);
      else ring[slot] = load(wn, s + P - KS);
    });
    wp = wn;
    wn = group(g + 2 * G);
    const int par = it & 1;
    static_for<NT>([&](auto n) FS_INLINE {
      red[((par * NW + wave) * NT + n) * kWave + lane] = acc[n];
    });
    __syncthreads();
    static_for<NT>([&](auto n) FS_INLINE {
      if ((n + it) % NW == wave) {
        f32x4 z = red[((par * NW + 0) * NT + n) * kWave + lane];
        for (int w = 1; w < NW; ++w) z += red[((par * NW + w) * NT + n) * kWave + lane];
        const int row0 = g * 16 - a.shift;
        float zt = 0.0f;
        bool has = false;
        const bool plain = row0 >= 0 && row0 + 16 <= a.V &&
                           __ballot(loc[n] >= row0 && loc[n] < row0 + 16) == 0;
        fold_logits<1>([&](auto) FS_INLINE { return z; }, row0, a.V, loc[n], plain, inv_t[n], m[n],
                       s_[n], zt, has);
        if (has) a.target[n * 16 + li] = zt;
      }
    });
  }
  __shared__ float2 fin[NW][NT * 16];
  static_for<NT>([&](auto n) FS_INLINE {
    pair_xor(m[n], s_[n], 16);
    pair_xor(m[n], s_[n], 32);
    if (kb == 0) fin[wave][n * 16 + li] = float2{m[n], s_[n]};
  });
  __syncthreads();
  const int c = threadIdx.x;
  if (c < NT * 16 && c < a.B) {
    float2 p = fin[0][c];
#pragma unroll
    for (int w = 1; w < NW; ++w) pair_merge(p.x, p.y, fin[w][c].x, fin[w][c].y);
    a.part[static_cast<size_t>(blockIdx.x) * a.B + c] = p;
  }
}

// ---------------------------------------------------------------------------
// The partials of each token into its log-probability and log-sum-exp.  A
// block takes COLS tokens; its threads split the S partials, eight loads of
// each in flight: bound by latency (4 to 8 us).
// ---------------------------------------------------------------------------
constexpr int kCloseThreads = 1024;

template <int COLS>
__global__ __launch_bounds__(kCloseThreads) void score_close_kernel(ScoreArgs a, float* logprob,
                                                                    float* lse) {
  constexpr int kSplit = kCloseThreads / COLS, kUnroll = 8;
  __shared__ float2 red[kSplit][COLS];
  const int c = threadIdx.x % COLS, y = threadIdx.x / COLS;
  const int b = blockIdx.x * COLS + c, bc = min(b, a.B - 1);
  float m = LseAcc::kMasked, s = 0.0f;
  for (int t0 = y; t0 < a.S; t0 += kSplit * kUnroll) {
    float2 p[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = t0 + u * kSplit;
      p[u] = t < a.S ? a.part[static_cast<size_t>(t) * a.B + bc] : float2{LseAcc::kMasked, 0.0f};
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) pair_merge(m, s, p[u].x, p[u].y);
  }
  red[y][c] = float2{m, s};
  __syncthreads();
#pragma unroll
  for (int k = kSplit / 2; k >= 1; k >>= 1) {
    if (y < k) {
      float2 p = red[y][c];
      pair_merge(p.x, p.y, red[y + k][c].x, red[y + k][c].y);
      red[y][c] = p;
    }
    __syncthreads();
  }
  if (y != 0 || b >= a.B) return;
  const float2 p = red[0][c];
  const int32_t id = a.ids[b];
  // log-sum-exp of the rows other than the target (-inf where there are none)
  const float rest = p.y == 0.0f ? -INFINITY : p.x + logf(p.y);
  if (target_row(id, a.vocab_offset, a.V) >= 0) {
    const float zt = a.target[b], x = rest - zt;
    const float soft = fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
    // NaN logits give NaN (fmaxf alone would drop it)
    logprob[b] = x != x ? x : -soft;
    // (a target at -inf: the others' alone)
    lse[b] = x != x ? x : zt == -INFINITY ? rest : zt + soft;
  } else {
    logprob[b] = id < 0 ? 0.0f : -INFINITY;
    lse[b] = rest;
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int32_t kMaxScoreB = 1 << 24;
constexpr int32_t kMaxScoreD = 1 << 20;
constexpr int kMaxStreamBlocks = 2048;

int64_t grid_tiles(int32_t B, int64_t S, int TB) { return (S * ((B + TB - 1) / TB) + 7) / 8 * 8; }

template <class T>
hipError_t launch_tile(ScoreArgs& a, hipStream_t stream) {
  static_assert(T::kThreads == (T::TA == kTallRows ? 512 : 256), "threads_of");
  a.S = static_cast<int32_t>((static_cast<int64_t>(a.V) + a.shift + T::TA - 1) / T::TA);
  static SmemRaised raised;
  const hipError_t e = raise_smem(&score_tile_kernel<T>, T::kSmemBytes, raised);
  if (e != hipSuccess) return e;
  score_tile_kernel<T><<<static_cast<unsigned>(grid_tiles(a.B, a.S, T::TB)), T::kThreads,
                         T::kSmemBytes, stream>>>(a);
  return hipGetLastError();
}

template <int L, bool NTA>
hipError_t launch_tiles(ScoreArgs& a, LogitsTile tile, hipStream_t stream) {
  switch (tile) {
    case LogitsTile::kTall64: return launch_tile<typename TallTile<L, 64, NTA>::T>(a, stream);
    case LogitsTile::kTall128: return launch_tile<typename TallTile<L, 128, NTA>::T>(a, stream);
    case LogitsTile::kTall256: return launch_tile<typename TallTile<L, 256>::T>(a, stream);
    case LogitsTile::kShort64: return launch_tile<typename ShortTile<L, 64, NTA>::T>(a, stream);
    case LogitsTile::kShort128: return launch_tile<typename ShortTile<L, 128, NTA>::T>(a, stream);
    default: return launch_tile<typename ShortTile<L, 256>::T>(a, stream);
  }
}

// Tokens of one tile read W in fragment order once: past the caches.  More
// tokens find it there (1300 tokens on 50000 rows of 1024 by tiles of 128: 154
// us through the caches, 177 past them).
template <int L>
hipError_t launch_tiles(ScoreArgs& a, hipStream_t stream) {
  const LogitsTile tile = logits_tile(a.B, a.V);
  if constexpr (L == kFrag)
    if (a.B <= tokens_of(tile)) return launch_tiles<L, true>(a, tile, stream);
  return launch_tiles<L, false>(a, tile, stream);
}

template <int NT, int NW, int KS, int P, bool PACKED, bool WHOLE = false>
hipError_t launch_stream(ScoreArgs& a, hipStream_t stream) {
  if constexpr (!WHOLE)
    if (a.D == 32 * NW * KS) return launch_stream<NT, NW, KS, P, PACKED, true>(a, stream);
  const auto kernel = score_stream_kernel<NT, NW, KS, P, PACKED, WHOLE>;
  constexpr size_t smem = 2ull * NW * NT * kWave * sizeof(f32x4);
  static OccupancyCache cache;
  int slots = resident_blocks(kernel, NW * kWave, smem, cache);
  if (slots <= 0) return hipErrorInvalidDevice;
  slots = slots < kMaxStreamBlocks ? slots : kMaxStreamBlocks;
  const int ngroups = static_cast<int>((static_cast<int64_t>(a.V) + a.shift + 15) / 16);
  a.S = ngroups < slots ? ngroups : slots;
  kernel<<<a.S, NW * kWave, smem, stream>>>(a);
  return hipGetLastError();
}

// Streaming where the waves' slices of h fit in registers: fewer instructions
// and no barrier per k tile (16 rows on 128256 x 4096: 180 us streaming, 201 by
// tiles; fragment order 157 and 170; 32 rows 175 and 203, 161 and 170).
bool streams(int32_t B, int32_t D) { return (B <= 16 && D <= 8192) || (B <= 32 && D <= 5120); }

// Waves per block, k-steps per wave and loads ahead, by row length.  Row-major
// rows gain from loads of a whole group ahead (128256 x 4096, 16 rows: 16 ahead
// 180 us, 8 ahead 187; 151936 x 5120: 10 ahead by sixteen waves 270, 4 ahead by
// eight 283), fragment order, whose groups are contiguous, from more waves
// (128256 x 4096, 32 rows: sixteen 161, eight 169; one row 155 and 159).
template <bool PACKED>
hipError_t launch_score_stream(ScoreArgs& a, hipStream_t stream) {
  const int32_t B = a.B, D = a.D;
  if (B <= 16) {
    if (D <= 1024) return launch_stream<1, 8, 4, 4, PACKED>(a, stream);
    if (D <= 2048) return launch_stream<1, 8, 8, 8, PACKED>(a, stream);
    if (D <= 4096) {
      if constexpr (PACKED) return launch_stream<1, 16, 8, 4, PACKED>(a, stream);
      else return launch_stream<1, 8, 16, 16, PACKED>(a, stream);
    }
    if (D <= 5120) {
      if constexpr (PACKED) return launch_stream<1, 8, 20, 4, PACKED>(a, stream);
      else return launch_stream<1, 16, 10, 10, PACKED>(a, stream);
    }
    if (D <= 6144) return launch_stream<1, 8, 24, 8, PACKED>(a, stream);
    return launch_stream<1, 8, 32, 8, PACKED>(a, stream);
  }
  if (D <= 1024) return launch_stream<2, 8, 4, 4, PACKED>(a, stream);
  if (D <= 2048) return launch_stream<2, 8, 8, 8, PACKED>(a, stream);
  if (D <= 4096) {
    if constexpr (PACKED) return launch_stream<2, 16, 8, 4, PACKED>(a, stream);
    else return launch_stream<2, 8, 16, 8, PACKED>(a, stream);
  }
  return launch_stream<2, 8, 20, 4, PACKED>(a, stream);
}

// Most vocabulary tiles of a call (the grid is shifted by up to 3 rows).
int32_t tile_count(int32_t B, int32_t V) {
  const int rows = is_tall(logits_tile(B, V)) ? kTallRows : kMinTileRows;
  return static_cast<int32_t>((static_cast<int64_t>(V) + 3 + rows - 1) / rows);
}

bool pads(int32_t B, int32_t D) { return !streams(B, D) && D % 64 != 0; }

struct ScoreLayout {
  size_t part, target, pad, total;
  ScoreLayout(int32_t B, int32_t D, int32_t V) {
    const size_t S = streams(B, D) ? kMaxStreamBlocks : tile_count(B, V);
    target = round_up(sizeof(float2) * S * B, 256);
    part = 0;
    pad = target + round_up(sizeof(float) * B, 256);
    total = pad + (pads(B, D) ? round_up(2 * static_cast<size_t>(B) * round_up(D, 64), 256) : 0);
  }
};

fs_status check_score_shape(const char* who, int32_t B, int32_t D, int32_t V,
                            int32_t vocab_offset) {
  if (B < 0) return fail(FS_ERR_INVALID_ARG, "%s: B must be >= 0 (got %d)", who, B);
  if (D < 8 || D % 8 != 0)
    return fail(FS_ERR_INVALID_ARG, "%s: D must be a positive multiple of 8 (got %d)", who, D);
  if (V < 1) return fail(FS_ERR_INVALID_ARG, "%s: V must be >= 1 (got %d)", who, V);
  if (vocab_offset < 0 || static_cast<int64_t>(vocab_offset) + V > 2147483647)
    return fail(FS_ERR_INVALID_ARG, "%s: vocab_offset and vocab_offset + V must be in [0, 2^31 - 1]"
                " (got %d, V = %d)", who, vocab_offset, V);
  if (B > kMaxScoreB || D > kMaxScoreD || V > kMaxVocab)
    return fail(FS_ERR_UNSUPPORTED, "%s: B=%d, D=%d, V=%d exceed the %d rows, %d elements or %d "
                "entries a call can take", who, B, D, V, kMaxScoreB, kMaxScoreD, kMaxVocab);
  if (!streams(B, D)) {  // (streaming grids are bounded by the device)
    const LogitsTile t = logits_tile(B, V);
    const int64_t S = (static_cast<int64_t>(V) + 3 + rows_of(t) - 1) / rows_of(t);
    if (!grid_fits(grid_tiles(B, S, tokens_of(t)), threads_of(t)))
      return fail(FS_ERR_UNSUPPORTED, "%s: B=%d, V=%d exceed the launch grid", who, B, V);
  }
  return FS_OK;
}

fs_status run_score(const char* who, const void* h, const void* W, int32_t B, int32_t D, int32_t V,
                    int32_t vocab_offset, const float* temperature, const int32_t* ids,
                    float* logprob, float* lse, void* workspace, size_t workspace_bytes,
                    void* stream, bool packed) {
  fs_status st = check_score_shape(who, B, D, V, vocab_offset);
  if (st != FS_OK) return st;
  if (packed && D % 32 != 0)
    return fail(FS_ERR_INVALID_ARG, "%s: D must be a multiple of 32 (got %d)", who, D);
  if (B == 0) return FS_OK;
  if (!h || !W || !ids || !logprob || !lse || !workspace)
    return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (!aligned(h, 16) || !aligned(W, 16))
    return fail(FS_ERR_INVALID_ARG, "%s: h and W must be 16-byte aligned", who);
  if (!aligned(ids, 4) || !aligned(logprob, 4) || !aligned(lse, 4) ||
      (temperature && !aligned(temperature, 4)))
    return fail(FS_ERR_INVALID_ARG, "%s: per-row arrays must be 4-byte aligned", who);
  if (!aligned(workspace, 256))
    return fail(FS_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  const ScoreLayout lay(B, D, V);
  if (workspace_bytes < lay.total)
    return fail(FS_ERR_WORKSPACE, "%s: workspace of %zu bytes is below the %zu required", who,
                workspace_bytes, lay.total);
  if (start_launches()) return injected_failure(who);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  ScoreArgs a;
  a.B = B;
  a.D = D;
  a.V = V;
  a.vocab_offset = vocab_offset;
  a.shift = packed ? vocab_offset & 3 : 0;
  a.w = packed ? Operand{static_cast<const __bf16*>(W), 16ll * D,
                         static_cast<int32_t>(packed_groups(V, vocab_offset)), D}
               : Operand{static_cast<const __bf16*>(W), D, V, D};
  a.h = Operand{static_cast<const __bf16*>(h), D, B, D};
  a.temperature = temperature;
  a.ids = ids;
  a.part = reinterpret_cast<float2*>(ws + lay.part);
  a.target = reinterpret_cast<float*>(ws + lay.target);
  hipError_t e;
  if (streams(B, D)) {
    e = packed ? launch_score_stream<true>(a, s) : launch_score_stream<false>(a, s);
  } else {
    if (pads(B, D)) {
      const int32_t Dp = static_cast<int32_t>(round_up(D, 64));
      __bf16* hp = reinterpret_cast<__bf16*>(ws + lay.pad);
      pad_rows_kernel<<<2048, 256, 0, s>>>(a.h.p, B, D, Dp, hp);
      if ((e = hipGetLastError()) != hipSuccess) return hip_fail(e, "padding launch");
      a.h = Operand{hp, Dp, B, Dp};
    }
    e = packed ? launch_tiles<kFrag>(a, s) : launch_tiles<kKC>(a, s);
  }
  if (e != hipSuccess) return hip_fail(e, "log-probability launch");
  // wide rows of the partials for many tokens (8192 tokens on 32000 rows of 256:
  // the call 205 us, 210 by eight), many threads per token for few
  if (B >= 2048)
    score_close_kernel<64><<<(B + 63) / 64, kCloseThreads, 0, s>>>(a, logprob, lse);
  else
    score_close_kernel<8><<<(B + 7) / 8, kCloseThreads, 0, s>>>(a, logprob, lse);
  e = hipGetLastError();
  return e == hipSuccess ? FS_OK : hip_fail(e, "log-probability merge launch");
}

}  // namespace
}  // namespace fs

extern "C" {

FS_API size_t fs_token_logprobs_workspace_bytes(int32_t B, int32_t D, int32_t V) {
  if (B < 0 || D < 8 || D % 8 != 0 || V < 1 || B > fs::kMaxScoreB || D > fs::kMaxScoreD ||
      V > fs::kMaxVocab)
    return 0;
  return fs::ScoreLayout(B, D, V).total;
}

FS_API fs_status fs_token_logprobs(const void* h, const void* W, int32_t B, int32_t D, int32_t V,
                                   int32_t vocab_offset, const float* temperature,
                                   const int32_t* token_ids, float* out_logprob, float* out_lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  return fs::run_score("fs_token_logprobs", h, W, B, D, V, vocab_offset, temperature, token_ids,
                       out_logprob, out_lse, workspace, workspace_bytes, stream, false);
}

FS_API fs_status fs_token_logprobs_packed(const void* h, const void* W_packed, int32_t B, int32_t D,
                                          int32_t V, int32_t vocab_offset, const float* temperature,
                                          const int32_t* token_ids, float* out_logprob,
                                          float* out_lse, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  return fs::run_score("fs_token_logprobs_packed", h, W_packed, B, D, V, vocab_offset, temperature,
                       token_ids, out_logprob, out_lse, workspace, workspace_bytes, stream, true);
}

}  // extern "C"
