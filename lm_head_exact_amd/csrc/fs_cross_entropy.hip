// fs_cross_entropy.hip -- the softmax cross entropy of the LM head with its
// gradients (fs_cross_entropy): hidden states and W in, loss, dh and dW out.
//
// With z = W h, lse = log sum exp z, p = exp(z - lse), target y, smoothing s and
// the coefficient l of the penalty on the log-sum-exp, a row's loss is
//   (1 - s) (lse - z_y) + s (lse - mean z) + l lse^2
// and, with u the incoming gradient and lift = 1 + 2 l lse,
//   dz_v = u (lift p_v - s / V - [v = y] (1 - s)),   dh = dz W,   dW = dz^T h.
// lse - z_y is taken as log(1 + exp(L - z_y)) with L the log-sum-exp of the
// others, and p_y - 1 as expm1 of its negative: neither cancels where the target
// is nearly certain.  Rows without a target are dropped before the products.
//
// Three products of 2 B V D operations.  The gradient needs lse, which needs all
// of a row's logits; what the first product leaves is therefore kept in 16 bits, for
// up to kKeptBytes (beyond that the logits are made a second time, a slice of the
// vocabulary after the other, in a fourth product: 4096 rows of 4096 on 128256, three
// quarters with a target, 8.0 ms kept and 10.2 made twice; 16000 rows 42.1 and 54.0;
// 513 rows on a shard of 16032 x 8192 387 and 484 us; 4 rows on 1000 x 256 41 and 43).
// Many short rows take that fourth product too (keeps()).
// Kept is not z, which 16 bits would blur by percents of p, but exp(z - m) with m the
// largest logit of the row within one wave's 16 to 128 vocabulary rows, and m itself
// in fp32 on the side: with the pairs (m, sum) merged into lse, one pass over it makes
//   dz = u lift exp(m - lse) * kept - u s / V
// in bf16, in place.  fp16 with the largest value at 2^15: 11 bits down to 2^-29
// of it and a value of 2^-39 of it lost, so that the one rounding that shows is
// dz's to bf16, as in fs_token_logprobs_backward (bf16 would be rounded twice:
// 2.4e-3 of dz instead of 1.7e-3).
//
// 4096 rows of 4096 on 128256, three quarters with a target: logits 2.6 to 2.7 ms, dW
// 2.6, dh 2.4 (1.2 to 1.3 PFLOP/s each), scaling the kept exponentials 0.27 (5.8 TB/s),
// everything else 0.12.  1777 rows of 5120 on 151936, the loss alone: 1.9 ms for the
// 1333 rows that count.
#include <cmath>

#include "fs_grad.hpp"

namespace fs {
namespace {

// Bytes of kept exponentials in a call.
constexpr int64_t kKeptBytes = int64_t{4} << 30;
constexpr float kLog2e = 1.44269504088896341f;

struct XentArgs {
  GradArgs g;
  float2* part;   // [S][Bp]: (m, sum of exp(z - m)) of a wave's vocabulary rows, target left out
  float* zsum;    // [S][Bp]: sum of z there, or null (no smoothing)
  float* zt;      // [Bp]: the target's logit
  float4* rows;   // [Bp]: loss, lse - z_y and lse^2 of each row that has a target
  int32_t S, sub;  // partials, and vocabulary rows of one
  float smoothing, z_loss, grad_scale;
  int32_t mean;
  float* losses;  // [B]
  float* stats;   // [3]
};

// The incoming gradient of a row's loss.
__device__ __forceinline__ float upstream(const XentArgs& x, int n) {
  return x.mean ? x.grad_scale / static_cast<float>(n) : x.grad_scale;
}
// What smoothing takes from every dz of a row.
__device__ __forceinline__ float uniform_term(const XentArgs& x, float up) {
  return x.smoothing > 0.0f ? -x.smoothing / static_cast<float>(x.g.V) * up : 0.0f;
}

enum Mode { kStats, kKeep, kDirect };

// The logits of a tile of vocabulary rows by rows with a target, in registers.
//   kStats   the pairs alone
//   kKeep    the pairs, and exp(z - m) in fp16
//   kDirect  dz, from the rows' terms
// A wave's maximum comes first (its logits are all in registers), then one
// exponential per logit, which goes to the sum in fp32 and out through LDS.
template <class T, int MODE>
__global__ __launch_bounds__(T::kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void xent_logits_kernel(XentArgs x) {
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn_smem[];
  const GradArgs& a = x.g;
  const int n = *a.count;
  int tile, btile;
  if (!xcd_tile<4>(blockIdx.x, (a.nv + T::TA - 1) / T::TA, (n + T::TB - 1) / T::TB, tile, btile))
    return;
  const int a0 = tile * T::TA, b0 = btile * T::TB;
  const Operand w = {a.W + static_cast<size_t>(a.v0) * a.D, a.D, a.nv, a.D};
  const Operand h = {a.hz, a.Dp, a.Bp, a.Dp};
  f32x4 acc[T::MR][T::NT];
  T::run(w, h, a0, b0, 0, a.Dp / T::BK, acc, dyn_smem);

  const int lane = threadIdx.x & (kWave - 1), li = lane & 15, kb = lane >> 4;
  const int wave_row = a0 + T::wave_a(), row0 = wave_row + 4 * kb;  // in the slice
  const bool whole = wave_row + T::MR * 16 <= a.nv;
  int loc[T::NT];
  static_for<T::NT>([&](auto n) FS_INLINE {
    loc[n] = a.loc[b0 + T::wave_b() + 16 * static_cast<int>(n) + li] - a.v0;
  });
  __bf16* out = a.dz + static_cast<size_t>(b0 + T::wave_b()) * a.ldz + wave_row;
  auto out_row = [&](int r) FS_INLINE { return out + static_cast<size_t>(r) * a.ldz; };
  auto keep_all = [&](int, int) FS_INLINE { return true; };

  if constexpr (MODE == kDirect) {
    const float uniform = uniform_term(x, upstream(x, n));
    const bool full = b0 + T::TB <= n;
    bool fill[T::NT];  // behind the last place: dz is 0 whatever the product with h = 0 gave
    RowTerm term[T::NT];
    static_for<T::NT>([&](auto nc) FS_INLINE {
      const int b = b0 + T::wave_b() + 16 * static_cast<int>(nc) + li;
      term[nc] = a.term[b];
      fill[nc] = !full && b >= n;
    });
    T::store_rows(
        dyn_smem,
        [&](auto m, auto nc) FS_INLINE {
          constexpr int n = decltype(nc)::value;
          const f32x4 z = acc[m][n];
          float d[4];
          static_for<4>([&](auto rc) FS_INLINE {
            constexpr int r = decltype(rc)::value;
            const int v = row0 + 16 * static_cast<int>(m) + r;
            const float p = __builtin_amdgcn_exp2f((z[r] - term[n].lse) * kLog2e);
            d[r] = __builtin_fmaf(p, term[n].coef, uniform);
            d[r] = v == loc[n] || (!whole && v >= a.nv) || fill[n] ? 0.0f : d[r];
          });
          return pack_bf16(d[0], d[1], d[2], d[3]);
        },
        out_row, keep_all);
    return;
  }

  float mz[T::NT], s[T::NT];
  bool plain[T::NT];  // the same on all lanes: no row of the wave is left out of any token's sum
  const size_t at = static_cast<size_t>((a.v0 + wave_row) / x.sub) * a.Bp + b0 + T::wave_b();
  static_for<T::NT>([&](auto n) FS_INLINE {
    const bool hit = loc[n] >= wave_row && loc[n] < wave_row + T::MR * 16;
    plain[n] = whole && __ballot(hit) == 0;
    float m = LseAcc::kMasked, zs = 0.0f;
    if (plain[n]) {
      static_for<T::MR>([&](auto i) FS_INLINE {
        const f32x4 z = acc[i][n];
        m = fmaxf(fmaxf(m, fmaxf(z[0], z[1])), fmaxf(z[2], z[3]));
      });
    } else {
      static_for<T::MR>([&](auto i) FS_INLINE {
        static_for<4>([&](auto r) FS_INLINE {
          const int v = row0 + 16 * static_cast<int>(i) + static_cast<int>(r);
          const float z = acc[i][n][decltype(r)::value];
          if (v == loc[n] && v < a.nv) x.zt[b0 + T::wave_b() + 16 * static_cast<int>(n) + li] = z;
          m = v < a.nv && v != loc[n] ? fmaxf(m, z) : m;
        });
      });
    }
    if (x.zsum != nullptr) {
      static_for<T::MR>([&](auto i) FS_INLINE {
        static_for<4>([&](auto r) FS_INLINE {
          const int v = row0 + 16 * static_cast<int>(i) + static_cast<int>(r);
          zs += whole || v < a.nv ? acc[i][n][decltype(r)::value] : 0.0f;
        });
      });
      zs += __shfl_xor(zs, 16, kWave);
      zs += __shfl_xor(zs, 32, kWave);
      if (kb == 0) x.zsum[at + 16 * static_cast<int>(n) + li] = zs;
    }
    m = fmaxf(m, __shfl_xor(m, 16, kWave));
    m = fmaxf(m, __shfl_xor(m, 32, kWave));
    mz[n] = m;
    s[n] = 0.0f;
  });
  // the exponentials of accumulator (m, n)
  auto exps = [&](auto m, auto nc, float (&e)[4]) FS_INLINE {
    constexpr int n = decltype(nc)::value;
    const f32x4 z = acc[m][n];
    static_for<4>([&](auto rc) FS_INLINE {
      constexpr int r = decltype(rc)::value;
      // (the difference first: it holds for logits of any size)
      e[r] = __builtin_amdgcn_exp2f(
          __builtin_fmaf(z[r] - mz[n], kLog2e, MODE == kKeep ? 15.0f : 0.0f));
    });
    if (!plain[n]) {
      static_for<4>([&](auto rc) FS_INLINE {
        constexpr int r = decltype(rc)::value;
        const int v = row0 + 16 * static_cast<int>(m) + r;
        e[r] = v < a.nv && v != loc[n] ? e[r] : 0.0f;
      });
    }
    s[n] += (e[0] + e[1]) + (e[2] + e[3]);
  };
  if constexpr (MODE == kKeep) {
    T::store_rows(
        dyn_smem,
        [&](auto m, auto n) FS_INLINE {
          typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
          float e[4];
          exps(m, n, e);
          return __builtin_bit_cast(
              uint64_t, f16x4{static_cast<_Float16>(e[0]), static_cast<_Float16>(e[1]),
                              static_cast<_Float16>(e[2]), static_cast<_Float16>(e[3])});
        },
        out_row, keep_all);
  } else {
    static_for<T::NT>([&](auto n) FS_INLINE {
      static_for<T::MR>([&](auto m) FS_INLINE {
        float e[4];
        exps(m, n, e);
      });
    });
  }
  static_for<T::NT>([&](auto n) FS_INLINE {
    s[n] += __shfl_xor(s[n], 16, kWave);
    s[n] += __shfl_xor(s[n], 32, kWave);
    if (MODE == kKeep) s[n] *= 0x1p-15f;
    if (kb == 0) x.part[at + 16 * static_cast<int>(n) + li] = float2{mz[n], s[n]};
  });
}

// ---------------------------------------------------------------------------
// The pairs of each row with a target into its loss and the terms of its
// gradient; the loss of the others is 0.  A block takes COLS places; its threads
// split the S pairs, eight loads of each in flight.
// ---------------------------------------------------------------------------
constexpr int kCloseThreads = 1024;

// ROWS: the partials are those of all rows in their own order (no gradient).
template <int COLS, bool ROWS>
__global__ __launch_bounds__(kCloseThreads) void xent_close_kernel(XentArgs x) {
  constexpr int kSplit = kCloseThreads / COLS, kUnroll = 8;
  __shared__ float2 red[kSplit][COLS];
  __shared__ double red_z[kSplit][COLS];
  const GradArgs& a = x.g;
  const int n = ROWS ? a.B : *a.count, ld = ROWS ? a.B : a.Bp;
  const int c = threadIdx.x % COLS, y = threadIdx.x / COLS;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * COLS + c;
  if (!ROWS && y == 0 && p < a.B && a.slot[p] < 0) x.losses[p] = 0.0f;  // (p is a row here)
  if (static_cast<int64_t>(blockIdx.x) * COLS >= n) return;     // (block-uniform)
  const int64_t pc = p < n ? p : n - 1;
  float m = LseAcc::kMasked, s = 0.0f;
  double zs = 0.0;
  for (int t0 = y; t0 < x.S; t0 += kSplit * kUnroll) {
    float2 q[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = t0 + u * kSplit;
      q[u] = t < x.S ? x.part[static_cast<size_t>(t) * ld + pc] : float2{LseAcc::kMasked, 0.0f};
    }
    if (x.zsum != nullptr) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int t = t0 + u * kSplit;
        zs += t < x.S ? x.zsum[static_cast<size_t>(t) * ld + pc] : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) pair_merge(m, s, q[u].x, q[u].y);
  }
  red[y][c] = float2{m, s};
  red_z[y][c] = zs;
  __syncthreads();
#pragma unroll
  for (int k = kSplit / 2; k >= 1; k >>= 1) {
    if (y < k) {
      float2 q = red[y][c];
      pair_merge(q.x, q.y, red[y + k][c].x, red[y + k][c].y);
      red[y][c] = q;
      red_z[y][c] += red_z[y + k][c];
    }
    __syncthreads();
  }
  if (y != 0 || p >= n) return;
  if (ROWS && !has_token(a.ids[p])) {
    x.losses[p] = 0.0f;
    x.rows[p] = float4{0.0f, 0.0f, 0.0f, 0.0f};
    return;
  }
  const float2 q = red[0][c];
  // log-sum-exp of the rows other than the target (-inf where there are none)
  const float rest = q.y == 0.0f ? -INFINITY : q.x + logf(q.y);
  const bool here = (ROWS ? target_row(a.ids[p], 0, a.V) : a.loc[p]) >= 0;
  float nll = INFINITY, lse = rest;  // a target past V has probability 0
  if (here) close_target(rest, x.zt[p], nll, lse);
  const float sm = x.smoothing;
  float loss = nll, own = 0.0f;
  const float lift = x.z_loss > 0.0f ? 1.0f + 2.0f * x.z_loss * lse : 1.0f;
  if (sm > 0.0f)  // (at 1 the target does not count, not even one of probability 0)
    loss = (sm < 1.0f ? (1.0f - sm) * nll : 0.0f) +
           sm * (lse - static_cast<float>(red_z[0][c] / a.V));
  if (x.z_loss > 0.0f) loss += x.z_loss * lse * lse;
  if (here) {
    own = expm1f(-nll);
    if (x.z_loss > 0.0f) own += 2.0f * x.z_loss * lse * expf(-nll);
    if (sm > 0.0f) own += sm * (1.0f - 1.0f / static_cast<float>(a.V));
  }
  x.losses[ROWS ? p : a.row[p]] = loss;
  x.rows[p] = float4{loss, nll, lse * lse, 1.0f};
  if (ROWS) return;
  const float up = upstream(x, n);
  a.term[p] = RowTerm{1.0f, lse, up * lift, up * own};
}

// The loss and the two means over the rows with a target, in a fixed order by
// one block.
template <int THREADS, bool ROWS>
__device__ void sum_rows(const XentArgs& x) {
  __shared__ double red[4][THREADS];
  const int places = ROWS ? x.g.B : *x.g.count, t = threadIdx.x;
  double v[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int64_t p = t; p < places; p += THREADS) {
    const float4 r = x.rows[p];
    v[0] += r.x;
    v[1] += r.y;
    v[2] += r.z;
    v[3] += r.w;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[i][t] = v[i];
  __syncthreads();
#pragma unroll
  for (int k = THREADS / 2; k >= 1; k >>= 1) {
    if (t < k)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[i][t] += red[i][t + k];
    __syncthreads();
  }
  if (t < 3)
    x.stats[t] = static_cast<float>(red[t][0] / (t == 0 && !x.mean ? 1.0 : fmax(red[3][0], 1.0)));
}

template <bool ROWS>
__global__ __launch_bounds__(1024) void xent_stats_kernel(XentArgs x) { sum_rows<1024, ROWS>(x); }

// Kept exponentials of one slice into dz, in place: 16 places by 1024 vocabulary
// rows per block (of 64 places 513 rows on a shard filled half the CUs).  Each
// place's factors for the block's partials are made once, in LDS; two waves then
// take a row, 16 bytes per lane.  The places that fill the last k tile of dW are set
// to 0: theirs are of h = 0, NaN where a row of W has an infinite entry.  Bound by
// reading and writing dz (4096 rows of 128256, three quarters with a target: 1.6 GB).
// The first slice's grid has one block more per column, the first of which makes the
// stats.
constexpr int kScaleRows = 16, kScaleCols = 1024;

__global__ __launch_bounds__(256) void xent_scale_kernel(XentArgs x) {
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  __shared__ float s_fac[kScaleCols / 16][kScaleRows];
  const GradArgs& a = x.g;
  if (a.first_slice && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) sum_rows<256, false>(x);
    return;
  }
  const int n = *a.count;
  const int r0 = blockIdx.x * kScaleRows, c0 = blockIdx.y * kScaleCols;
  if (r0 >= (n + kGradPlaces - 1) / kGradPlaces * kGradPlaces) return;
  const int lane_col = (threadIdx.x % 128) * 8, c = c0 + lane_col, half = threadIdx.x / 128;
  const bool mine = c < (a.nv + 7) / 8 * 8;
  constexpr int kEach = kScaleRows / 2;  // rows of a thread
  u32x4* at = reinterpret_cast<u32x4*>(a.dz + static_cast<size_t>(r0 + half) * a.ldz + c);
  const size_t step = static_cast<size_t>(a.ldz) / 4;  // two rows
  f16x8 e[kEach];
  if (mine) {
#pragma unroll
    for (int u = 0; u < kEach; ++u)
      e[u] = __builtin_bit_cast(f16x8, __builtin_nontemporal_load(at + u * step));
  }
  {  // a thread's row of the factors is threadIdx.x mod 16
    const int r = threadIdx.x % kScaleRows, p = min(r0 + r, n - 1);
    const int t0 = c0 / x.sub, count = min((a.nv + x.sub - 1) / x.sub - t0, kScaleCols / x.sub);
    const RowTerm term = a.term[p];
    constexpr int kMost = kScaleCols / 16 * kScaleRows / 256;
    float m[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      const int t = min(static_cast<int>(threadIdx.x) / kScaleRows + k * (256 / kScaleRows), count - 1);
      m[k] = x.part[static_cast<size_t>(a.v0 / x.sub + t0 + t) * a.Bp + p].x;
    }
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      const int t = threadIdx.x / kScaleRows + k * (256 / kScaleRows);
      const float f =
          __builtin_amdgcn_exp2f((m[k] - term.lse) * kLog2e) * term.coef * 0x1p-15f;
      if (t < kScaleCols / x.sub) s_fac[t][r] = f;
    }
  }
  __syncthreads();
  if (!mine) return;
  const float uniform = uniform_term(x, upstream(x, n));
  const int fac = lane_col / x.sub;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int row = 2 * u + half, p = r0 + row;
    const float f = s_fac[fac][row];
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = p < n ? static_cast<float>(e[u][j]) * f : 0.0f;
    if (x.smoothing > 0.0f && p < n) {
      const int loc = a.loc[p] - a.v0;
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] += c + j < a.nv && c + j != loc ? uniform : 0.0f;
    }
    const uint64_t lo = pack_bf16(d[0], d[1], d[2], d[3]), hi = pack_bf16(d[4], d[5], d[6], d[7]);
    at[u * step] = u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                         static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Vocabulary rows of one wave of a tile.
int wave_rows(LogitsTile t) {
  switch (t) {
    case LogitsTile::kTall64: return TallTile<kKC, 64>::T::MR * 16;
    case LogitsTile::kTall128: return TallTile<kKC, 128>::T::MR * 16;
    case LogitsTile::kTall256: return TallTile<kKC, 256>::T::MR * 16;
    case LogitsTile::kShort64: return ShortTile<kKC, 64>::T::MR * 16;
    case LogitsTile::kShort128: return ShortTile<kKC, 128>::T::MR * 16;
    default: return ShortTile<kKC, 256>::T::MR * 16;
  }
}

// Where D is small and the rows many, the fourth product costs less than the memory
// that the kept exponentials pass through (4096 rows on 20000, us kept and made twice:
// D = 64 278 and 248, 128 292 and 266, 256 324 and 320, 384 365 and 380, 1024 605 and 696;
// of 300 rows on 30000, which the caches hold, kept wins from D = 64 on: 74 and 78).
bool keeps(int32_t B, int32_t D, int32_t V) {
  return (D > 256 || B <= 512) &&
         2 * static_cast<int64_t>(round_up(B, 256)) * static_cast<int64_t>(round_up(V, 256)) <=
             kKeptBytes;
}

// The loss alone of up to 128 rows, without smoothing: the partials of fs_token_logprobs'
// kernels, one pair per block, of all rows in their own order (one row on 128256 x 4096
// 175 us, 200 by this file's tiles; on 57749 x 3896 84 and 117; 128 rows 116 and 127).
// Beyond that, rows without a target are worth dropping first (160 rows on 128256 x
// 4096, 60% without: 261 and 208; 256 rows that all have one 269 and 283).
bool scores(int32_t B, int32_t D, int32_t V) { return B <= 128 && score_grid_fits(B, D, V); }

struct XentPlan {
  bool keep;
  GradPlan g;
  LogitsTile tile;
  int32_t S, sub;
  size_t part, zsum, zt, rows, total;
  // of scored rows: rows [B], then the partials
  static size_t rows_at(int32_t B) { return round_up(sizeof(float4) * B, 256); }
  XentPlan(int32_t B, int32_t D, int32_t V, bool grads)
      : keep(keeps(B, D, V)), g(B, D, V, keep, true) {
    tile = logits_tile(B, g.slice < V ? g.slice : V, true);
    sub = wave_rows(tile);
    // the last slice's tiles may end before it does
    const int64_t before = static_cast<int64_t>(g.slices - 1) * g.slice;
    S = static_cast<int32_t>((before + round_up(V - before, rows_of(tile))) / sub);
    size_t at = grads ? g.total : g.dz;  // (without gradients nothing behind the hidden states)
    auto take = [&](size_t bytes) {
      const size_t o = at;
      at += round_up(bytes, 256);
      return o;
    };
    part = take(sizeof(float2) * S * g.Bp);
    zsum = take(sizeof(float) * S * g.Bp);
    zt = take(sizeof(float) * g.Bp);
    rows = take(sizeof(float4) * g.Bp);
    total = at;
    if (!grads && scores(B, D, V)) total = std::max(total, rows_at(B) + ScoreLayout(B, D, V).total);
  }
};

template <class T, int MODE>
hipError_t launch_tile(const XentArgs& x, hipStream_t stream) {
  static SmemRaised raised;
  const hipError_t e = raise_smem(&xent_logits_kernel<T, MODE>, T::kSmemBytes, raised);
  if (e != hipSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((x.g.nv + T::TA - 1) / T::TA) *
                        ((x.g.B + T::TB - 1) / T::TB);
  xent_logits_kernel<T, MODE><<<static_cast<unsigned>((tiles + 7) / 8 * 8), T::kThreads,
                                T::kSmemBytes, stream>>>(x);
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_logits(const XentArgs& x, LogitsTile tile, hipStream_t stream) {
  switch (tile) {
    case LogitsTile::kTall64: return launch_tile<TallTile<kKC, 64>::T, MODE>(x, stream);
    case LogitsTile::kTall128: return launch_tile<TallTile<kKC, 128>::T, MODE>(x, stream);
    case LogitsTile::kTall256: return launch_tile<TallTile<kKC, 256>::T, MODE>(x, stream);
    case LogitsTile::kShort64: return launch_tile<ShortTile<kKC, 64>::T, MODE>(x, stream);
    case LogitsTile::kShort128: return launch_tile<ShortTile<kKC, 128>::T, MODE>(x, stream);
    default: return launch_tile<ShortTile<kKC, 256>::T, MODE>(x, stream);
  }
}

hipError_t launch_scale(const XentArgs& x, hipStream_t stream) {
  const int blocks = (x.g.B + kGradPlaces - 1) / kGradPlaces * (kGradPlaces / kScaleRows);
  const dim3 grid(blocks + (x.g.first_slice ? 1 : 0),
                  (x.g.nv + kScaleCols - 1) / kScaleCols);
  xent_scale_kernel<<<grid, 256, 0, stream>>>(x);
  return hipGetLastError();
}

hipError_t run_xent(XentArgs& x, const XentPlan& p, hipStream_t s) {
  GradArgs& a = x.g;
  const bool grads = a.dh != nullptr || a.dW != nullptr;
  __bf16* const dz = a.dz;
  // slice i of the vocabulary; kept exponentials lie one slice behind the other
  auto slice = [&](int i) {
    a.v0 = i * p.g.slice;
    a.nv = a.V - a.v0 < p.g.slice ? a.V - a.v0 : p.g.slice;
    a.first_slice = i == 0;
    a.dz = dz + (p.keep ? static_cast<size_t>(i) * a.Bp * a.ldz : 0);
  };
  hipError_t e = launch_grad_rows(a, s);
  if (e != hipSuccess) return e;
  if (a.B > 0) {
    for (int i = 0; i < p.g.slices; ++i) {
      slice(i);
      e = grads && p.keep ? launch_logits<kKeep>(x, p.tile, s) : launch_logits<kStats>(x, p.tile, s);
      if (e != hipSuccess) return e;
    }
    if (a.B >= 2048) xent_close_kernel<64, false><<<(a.B + 63) / 64, kCloseThreads, 0, s>>>(x);
    else xent_close_kernel<8, false><<<(a.B + 7) / 8, kCloseThreads, 0, s>>>(x);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (!grads || !p.keep || a.B == 0) {
    xent_stats_kernel<false><<<1, 1024, 0, s>>>(x);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (!grads) return hipSuccess;
  for (int i = 0; i < p.g.slices; ++i) {
    slice(i);
    if (a.B > 0) e = p.keep ? launch_scale(x, s) : launch_logits<kDirect>(x, p.tile, s);
    if (e != hipSuccess) return e;
    if ((e = launch_grad_products(a, s)) != hipSuccess) return e;
  }
  return launch_grad_finish(a, s);
}

hipError_t run_scored(XentArgs& x, char* ws, hipStream_t s) {
  GradArgs& a = x.g;
  const ScoreLayout lay(a.B, a.D, a.V);
  ScoreArgs c;
  c.w = Operand{a.W, a.D, a.V, a.D};
  c.h = Operand{a.h, a.D, a.B, a.D};
  c.B = a.B;
  c.D = a.D;
  c.V = a.V;
  c.vocab_offset = c.shift = 0;
  c.temperature = nullptr;
  c.ids = a.ids;
  hipError_t e = launch_score_logits(c, ws + XentPlan::rows_at(a.B), lay, false, s);
  if (e != hipSuccess) return e;
  x.rows = reinterpret_cast<float4*>(ws);
  x.part = c.part;
  x.zt = c.target;
  x.S = c.S;
  xent_close_kernel<8, true><<<(a.B + 7) / 8, kCloseThreads, 0, s>>>(x);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  xent_stats_kernel<true><<<1, 1024, 0, s>>>(x);
  return hipGetLastError();
}

}  // namespace
}  // namespace fs

extern "C" {

FS_API size_t fs_cross_entropy_workspace_bytes(int32_t B, int32_t D, int32_t V, int32_t grads) {
  return fs::grad_sizes_ok(B, D, V) ? fs::XentPlan(B > 0 ? B : 1, D, V, grads != 0).total : 0;
}

FS_API fs_status fs_cross_entropy(const void* h, const void* W, int32_t B, int32_t D, int32_t V,
                                  const int32_t* targets, double label_smoothing, double z_loss,
                                  int32_t mean, double grad_scale, float* out_stats,
                                  float* out_losses, void* grad_h, void* grad_W, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  using namespace fs;
  const char* who = "fs_cross_entropy";
  if (B < 0) return fail(FS_ERR_INVALID_ARG, "%s: B must be >= 0 (got %d)", who, B);
  if (D < 8 || D % 8 != 0)
    return fail(FS_ERR_INVALID_ARG, "%s: D must be a positive multiple of 8 (got %d)", who, D);
  if (V < 1) return fail(FS_ERR_INVALID_ARG, "%s: V must be >= 1 (got %d)", who, V);
  if (!grad_sizes_ok(B, D, V))
    return fail(FS_ERR_UNSUPPORTED, "%s: B=%d, D=%d, V=%d exceed the %d rows, %d elements or %d "
                "entries a call can take", who, B, D, V, kMaxGradB, kMaxGradD, kMaxVocab);
  if (!(label_smoothing >= 0.0 && label_smoothing <= 1.0))
    return fail(FS_ERR_INVALID_ARG, "%s: label_smoothing must be in [0, 1] (got %g)", who,
                label_smoothing);
  if (!(z_loss >= 0.0) || !std::isfinite(z_loss))
    return fail(FS_ERR_INVALID_ARG, "%s: z_loss must be finite and >= 0 (got %g)", who, z_loss);
  if (!std::isfinite(grad_scale))
    return fail(FS_ERR_INVALID_ARG, "%s: grad_scale must be finite (got %g)", who, grad_scale);
  if (!W || !out_stats || (B > 0 && (!h || !targets || !out_losses)) || !workspace)
    return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(grad_h, 16) || !aligned(grad_W, 16))
    return fail(FS_ERR_INVALID_ARG, "%s: h, W and their gradients must be 16-byte aligned", who);
  if (!aligned(targets, 4) || !aligned(out_stats, 4) || !aligned(out_losses, 4))
    return fail(FS_ERR_INVALID_ARG, "%s: per-row arrays must be 4-byte aligned", who);
  if (!aligned(workspace, 256))
    return fail(FS_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  const XentPlan p(B > 0 ? B : 1, D, V, grad_h || grad_W);
  if (workspace_bytes < p.total)
    return fail(FS_ERR_WORKSPACE, "%s: workspace of %zu bytes is below the %zu required", who,
                workspace_bytes, p.total);
  if (!grad_grids_fit(B, D, V, p.g, B > 0 && grad_h, grad_W))
    return fail(FS_ERR_UNSUPPORTED, "%s: B=%d, D=%d, V=%d exceed the launch grid", who, B, D, V);
  if (start_launches()) return injected_failure(who);
  char* ws = static_cast<char*>(workspace);
  XentArgs x;
  GradArgs& a = x.g;
  a.h = static_cast<const __bf16*>(h);
  a.W = static_cast<const __bf16*>(W);
  a.B = B;
  a.D = D;
  a.V = V;
  a.vocab_offset = 0;
  a.temperature = a.logprob = a.lse = a.grad = nullptr;
  a.ids = targets;
  a.dh = B > 0 ? static_cast<__bf16*>(grad_h) : nullptr;
  a.dW = static_cast<__bf16*>(grad_W);
  grad_workspace(a, p.g, ws);
  x.part = reinterpret_cast<float2*>(ws + p.part);
  x.zsum = label_smoothing > 0.0 ? reinterpret_cast<float*>(ws + p.zsum) : nullptr;
  x.zt = reinterpret_cast<float*>(ws + p.zt);
  x.rows = reinterpret_cast<float4*>(ws + p.rows);
  x.S = p.S;
  x.sub = p.sub;
  x.smoothing = static_cast<float>(label_smoothing);
  x.z_loss = static_cast<float>(z_loss);
  x.grad_scale = static_cast<float>(grad_scale);
  x.mean = mean != 0;
  x.losses = out_losses;
  x.stats = out_stats;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool scored = !a.dh && !a.dW && B > 0 && !x.zsum && scores(B, D, V);
  const hipError_t e = scored ? run_scored(x, ws, s) : run_xent(x, p, s);
  return e == hipSuccess ? FS_OK : hip_fail(e, "cross-entropy launch");
}

}  // extern "C"
