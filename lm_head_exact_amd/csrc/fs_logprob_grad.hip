// fs_logprob_grad.hip -- gradients of token log-probabilities with respect to
// the hidden states and the LM head (fs_token_logprobs_backward).
//
// With t = z * fp32(1/T) the scaled logits, p_v = exp(t_v - lse) and g the
// incoming gradient of a row's log-probability,
//   dz_v = g/T * ( [v = target] (1 - p_target) - [v != target] p_v )
//   dh = dz W,   dW = dz^T h
// 1 - p_target is -expm1(logprob) of the forward pass: from p itself it would
// be noise where the target is nearly certain.  Rows without a target (prompt
// or padding tokens) have no gradient: they are dropped before the products,
// so they cost nothing and NaN in their hidden states stays there.
//
// dz (B x V) is made in bf16, one slice of the vocabulary at a time, from the
// logits recomputed on chip, and both products read it back from the
// workspace.  MFMA takes bf16 operands, so every dz is rounded once (by up to
// 2^-8 of it, 1.7e-3 root mean square), but for the targets': they are what most of a gradient is made
// of, a rounding of them would not average out, and there is one per row.  dz
// holds zero there, and their terms are added in fp32 where the results are
// rounded: g/T (1 - p) W_target to a row of dh, g/T (1 - p) h to a target's
// row of dW (the product leaves those rows in fp32 on the side).  Measured
// against fp64 (Frobenius norm): 1.7e-3 with 2.4e-3 before, bf16 results alone
// being 1.7e-3; up to 2.0e-3 where few of the batch's targets lie in the rows of
// W.  (A second bf16 for what the first leaves would halve the rate of both
// products.)
//
// Three matrix products of 2 B V D operations each bound the call for batches
// of training; a batch of a few rows is bound by reading W twice and writing
// dW.  4096 tokens, of which three quarters count, on 128256 rows of 4096:
// logits 2.4 to 2.8 ms, dW 2.5 to 2.7, dh 2.4 to 2.5 (1.2 to 1.3 PFLOP/s each),
// everything else 0.11 ms.  One token there: 175, 230 and 168 us (6.0, 4.6 and 6.2 TB/s).
#include <algorithm>
#include <cmath>

#include "fs_host.hpp"
#include "fs_score.hpp"
#include "fs_sampler.hpp"

namespace fs {
namespace {

// Per row that has a target, in order.
struct RowTerm {
  float c;       // log2(e) / T
  float lse2;    // log2(e) * lse
  float coef;    // -g / T
  float target;  // g / T * (1 - p_target)
};

struct GradArgs {
  const __bf16 *h, *W;
  int32_t B, D, V, vocab_offset;
  const float *temperature, *logprob, *lse, *grad;
  const int32_t* ids;
  __bf16 *dh, *dW;    // either may be null
  // workspace
  int32_t* count;     // [2]: rows with a target; parts of the vocabulary for dh
  int32_t* slot;      // [B]: their place among them, or -1
  int32_t* row;       // [Bp]: the inverse
  int32_t* loc;       // [Bp]: target's row of W, or -1
  RowTerm* term;      // [Bp]
  __bf16* hz;         // [Bp][Dp]: their hidden states, zeros behind them
  __bf16* dz;         // [Bp][ldz]
  float* slab;        // [max_splits][B][D] or null
  // targets by tile of 256 vocabulary rows
  int32_t* first;     // [V]: first place whose target the row is, or -1
  int32_t* list;      // [Bp]: places that have a target here, by tile
  int2* tile;         // [tiles]: begin and end in `list`
  float* side;        // [Bp][D]: dW rows of targets, at their first place
  int32_t Dp, Bp, ldz;
  int32_t v0, nv;     // the slice: rows v0 .. v0 + nv of W
  int32_t max_splits, hidden_tb, first_slice;
};

// A row counts where it has a token; a token of another shard still gives
// every row of this one a gradient.
__device__ __forceinline__ bool has_token(int32_t id) { return id >= 0; }

constexpr int kScanThreads = 1024;

// Estimated time of dh over `parts` parts of a slice's vocabulary rows, in k
// tiles of 64: rounds of blocks over the CUs, each its share of the k tiles
// and about six of prologue and epilogue, and for every part a slab of fp32
// written and read (8e5 of its elements take about as long as one k tile).
__device__ __forceinline__ uint64_t hidden_cost(const GradArgs& a, int n, int parts) {
  constexpr int kCus = 256;
  const int nk = a.ldz / 64;
  const uint64_t tiles =
      static_cast<uint64_t>((n + a.hidden_tb - 1) / a.hidden_tb) * ((a.D + 255) / 256);
  return (tiles * parts + kCus - 1) / kCus * ((nk + parts - 1) / parts + 6) +
         static_cast<uint64_t>(parts) * n * a.D / 800000;
}

// Places of the rows that have a token, in order (one block), and the parts of
// the vocabulary that dh is taken in: its tiles alone are few, and rows without
// a token leave some of them empty, so that whole rounds of tiles would leave
// many CUs idle.  The same number for every slice of a call, so that each adds
// to the same slabs.  One block, 3 us and 1 us per thousand rows: the rows'
// order needs a scan, and the host does not know how many count.
__global__ __launch_bounds__(kScanThreads) void grad_rows_kernel(GradArgs a) {
  constexpr int kWaves = kScanThreads / kWave;
  __shared__ int32_t s[kWaves];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  int base = 0;
  for (int64_t b0 = 0; b0 < a.B; b0 += kScanThreads) {
    const int64_t b = b0 + threadIdx.x;
    const bool on = b < a.B && has_token(a.ids[b]);
    const uint64_t votes = __ballot(on);
    if (lane == 0) s[wave] = __popcll(votes);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      before += w < wave ? s[w] : 0;
      all += s[w];
    }
    const int at = base + before + __popcll(votes & ((uint64_t{1} << lane) - 1));
    if (b < a.B) {
      a.slot[b] = on ? at : -1;
      if (on) a.row[at] = static_cast<int32_t>(b);
    }
    base += all;
    __syncthreads();
  }
  __shared__ unsigned long long best;
  if (threadIdx.x == 0) best = ~0ull;
  __syncthreads();
  const int parts = static_cast<int>(threadIdx.x) + 1;  // the least cost, then the fewest parts
  unsigned long long cost = parts <= a.max_splits ? hidden_cost(a, base, parts) << 12 | parts : ~0ull;
#pragma unroll
  for (int m = kWave / 2; m >= 1; m >>= 1)
    cost = min(cost, static_cast<unsigned long long>(__shfl_xor(cost, m, kWave)));
  if (lane == 0) atomicMin(&best, cost);
  __syncthreads();
  if (threadIdx.x == 0) {
    a.count[0] = base;
    a.count[1] = static_cast<int32_t>(best & 4095);
  }
}

// Row b < B: its terms and a copy of its hidden state at its place, or a zero
// gradient.  Rows B .. B + 255: zeros up to the next multiple of 256 places.
// Copies 64 MB (4096 rows of 4096, read and written) in 12 us.
__global__ __launch_bounds__(256) void grad_gather_kernel(GradArgs a) {
  const int b = blockIdx.x;
  const int n = *a.count;
  int at;
  if (b < a.B) {
    at = a.slot[b];
    if (at < 0) {
      if (a.dh != nullptr)
        for (int k = threadIdx.x * 8; k < a.D; k += 256 * 8)
          *reinterpret_cast<bf16x8*>(a.dh + static_cast<size_t>(b) * a.D + k) = zero_frag();
      return;
    }
    for (int k = threadIdx.x * 8; k < a.Dp; k += 256 * 8)
      *reinterpret_cast<bf16x8*>(a.hz + static_cast<size_t>(at) * a.Dp + k) =
          k < a.D ? load_frag(a.h + static_cast<size_t>(b) * a.D + k) : zero_frag();
  } else {
    at = n + (b - a.B);
    if (at >= (n + 255) / 256 * 256) return;
    for (int k = threadIdx.x * 8; k < a.Dp; k += 256 * 8)
      *reinterpret_cast<bf16x8*>(a.hz + static_cast<size_t>(at) * a.Dp + k) = zero_frag();
  }
  if (threadIdx.x != 0) return;
  RowTerm t = {0.0f, 0.0f, 0.0f, 0.0f};
  int loc = -1;
  if (b < a.B) {
    const float inv_t = score_inv_t(a.temperature, b);
    const float g = a.grad[b] * inv_t;
    t.c = inv_t * 1.44269504088896341f;
    t.lse2 = a.lse[b] * 1.44269504088896341f;
    t.coef = -g;
    loc = target_row(a.ids[b], a.vocab_offset, a.V);
    t.target = loc >= 0 ? -expm1f(a.logprob[b]) * g : 0.0f;
  }
  a.term[at] = t;
  a.loc[at] = loc;
}

__device__ __forceinline__ uint64_t pack_bf16(float x0, float x1, float x2, float x3) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  const bf16x4 v = {static_cast<__bf16>(x0), static_cast<__bf16>(x1), static_cast<__bf16>(x2),
                    static_cast<__bf16>(x3)};
  return __builtin_bit_cast(uint64_t, v);
}

// The places that have a target in one tile of 256 vocabulary rows, in order,
// and each row's first one.  Every block reads all targets, twice: B ints
// against the B * 256 * D products of the tile (3 to 6 us).
constexpr int kTargetTile = 256;
constexpr int kTargetThreads = 1024;

__global__ __launch_bounds__(kTargetThreads) void grad_targets_kernel(GradArgs a) {
  constexpr int kWaves = kTargetThreads / kWave;
  __shared__ int32_t s_before[kWaves], s_in[kWaves];
  __shared__ int32_t s_first[kTargetTile];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int lo = static_cast<int>(blockIdx.x) * kTargetTile;
  const int64_t n = *a.count;
  const int p0 = static_cast<int>(n * wave / kWaves), p1 = static_cast<int>(n * (wave + 1) / kWaves);
  if (threadIdx.x < kTargetTile) s_first[threadIdx.x] = 0x7FFFFFFF;
  int before = 0, in = 0;
#pragma unroll 8
  for (int p = p0 + lane; p < p1; p += kWave) {
    const int l = a.loc[p];
    before += l >= 0 && l < lo;
    in += l >= lo && l - lo < kTargetTile;
  }
#pragma unroll
  for (int m = kWave / 2; m >= 1; m >>= 1) {
    before += __shfl_xor(before, m, kWave);
    in += __shfl_xor(in, m, kWave);
  }
  if (lane == 0) {
    s_before[wave] = before;
    s_in[wave] = in;
  }
  __syncthreads();
  int begin = 0, at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    begin += s_before[w];
    at += w < wave ? s_in[w] : 0;
    all += s_in[w];
  }
  if (in > 0) {  // uniform per wave
    at += begin;
    for (int q = p0; q < p1; q += kWave) {
      const int p = q + lane;
      const int l = p < p1 ? a.loc[p] : -1;
      const bool hit = l >= lo && l - lo < kTargetTile;
      const uint64_t votes = __ballot(hit);
      if (hit) {
        a.list[at + __popcll(votes & ((uint64_t{1} << lane) - 1))] = p;
        atomicMin(&s_first[l - lo], p);  // (the minimum does not depend on the order)
      }
      at += __popcll(votes);
    }
  }
  __syncthreads();
  const int v = lo + static_cast<int>(threadIdx.x);
  if (threadIdx.x < kTargetTile && v < a.V)
    a.first[v] = s_first[threadIdx.x] == 0x7FFFFFFF ? -1 : s_first[threadIdx.x];
  if (threadIdx.x == 0) a.tile[blockIdx.x] = int2{begin, begin + all};
}

// dz of one slice: logits of a tile of vocabulary rows by rows with a target,
// turned into dz in registers: the product's tile loop and one exponential and
// store of 2 bytes per logit, which its own stores through LDS keep whole.
template <class T>
__global__ __launch_bounds__(T::kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void grad_logits_kernel(GradArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn_smem[];
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
  const int row0 = a0 + T::wave_a() + 4 * kb;  // in the slice
  const bool whole = a0 + T::TA <= a.nv;
  RowTerm term[T::NT];
  int loc[T::NT];
  static_for<T::NT>([&](auto n) FS_INLINE {
    const int b = b0 + T::wave_b() + 16 * static_cast<int>(n) + li;
    term[n] = a.term[b];
    loc[n] = a.loc[b] - a.v0;
  });
  __bf16* out = a.dz + static_cast<size_t>(b0 + T::wave_b()) * a.ldz + a0 + T::wave_a();
  T::store_rows(
      dyn_smem,
      [&](auto m, auto nc) FS_INLINE {
        constexpr int n = decltype(nc)::value;
        const f32x4 z = acc[m][n];
        float d[4];
        static_for<4>([&](auto rc) FS_INLINE {
          constexpr int r = decltype(rc)::value;
          const int v = row0 + 16 * static_cast<int>(m) + r;
          d[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[r], term[n].c, -term[n].lse2)) * term[n].coef;
          d[r] = v == loc[n] || (!whole && v >= a.nv) ? 0.0f : d[r];
        });
        return pack_bf16(d[0], d[1], d[2], d[3]);
      },
      [&](int r) FS_INLINE { return out + static_cast<size_t>(r) * a.ldz; },
      [&](int, int) FS_INLINE { return true; });
}

// dW of one slice: rows v of W, columns d, summed over the rows with a target.
template <class T>
__global__ __launch_bounds__(T::kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void grad_weights_kernel(GradArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn_smem[];
  const int n = *a.count;
  int tile, dtile;
  if (!xcd_tile<4>(blockIdx.x, (a.nv + T::TB - 1) / T::TB, (a.D + T::TA - 1) / T::TA, tile, dtile))
    return;
  const int a0 = dtile * T::TA, b0 = tile * T::TB;
  const Operand h = {a.hz, a.Dp, a.D, a.Bp};
  const Operand z = {a.dz, a.ldz, a.ldz, a.Bp};
  f32x4 acc[T::MR][T::NT];
  if (n > 0) T::run(h, z, a0, b0, 0, (n + T::BK - 1) / T::BK, acc, dyn_smem);
  else zero_acc(acc);
  const int lane = threadIdx.x & (kWave - 1), li = lane & 15, kb = lane >> 4;
  const int d0 = a0 + T::wave_a() + 4 * kb;
  // rows that are a target go to the side in fp32, the others to dW
  int place[T::NT];
  static_for<T::NT>([&](auto n) FS_INLINE {
    const int v = b0 + T::wave_b() + 16 * static_cast<int>(n) + li;
    place[n] = v < a.nv ? a.first[a.v0 + v] : -1;
  });
  static_for<T::NT>([&](auto n) FS_INLINE {
    if (place[n] >= 0) {
      float* side = a.side + static_cast<size_t>(place[n]) * a.D + d0;
      static_for<T::MR>([&](auto m) FS_INLINE {
        if (d0 + 16 * static_cast<int>(m) < a.D)
          *reinterpret_cast<f32x4*>(side + 16 * static_cast<int>(m)) = acc[m][n];
      });
    }
  });
  const int v0 = b0 + T::wave_b(), c0 = a0 + T::wave_a();
  __bf16* out = a.dW + (static_cast<size_t>(a.v0) + v0) * a.D + c0;
  T::template store_rows<true>(
      dyn_smem,
      [&](auto m, auto n) FS_INLINE {
        const f32x4 x = acc[m][n];
        return pack_bf16(x[0], x[1], x[2], x[3]);
      },
      [&](int r) FS_INLINE { return out + static_cast<size_t>(r) * a.D; },
      [&](int r, int c) FS_INLINE { return v0 + r < a.nv && c0 + c < a.D; });
}

// The targets' rows of dW: what the product left on the side plus each target's
// own term, in the order of the places, rounded once.  One block per place,
// which has something to do where it is its target's first; a thread takes
// eight columns.  The block looks through its tile's targets 256 at a time for
// those that are its own, then adds these.  9 us for 513 rows, 25 for 4096.
__global__ __launch_bounds__(256) void grad_target_rows_kernel(GradArgs a) {
  constexpr int kThreads = 256, kWaves = kThreads / kWave, kAhead = 8;
  __shared__ int32_t s_place[kThreads + kAhead];
  __shared__ int32_t s_count[kWaves];
  const int p = blockIdx.x;
  if (p >= a.count[0]) return;
  const int loc = a.loc[p];
  if (loc < 0 || a.first[loc] != p) return;
  const int2 range = a.tile[loc / kTargetTile];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  const int span = gridDim.y * kThreads * 8;
  for (int d0 = blockIdx.y * kThreads * 8; d0 < a.D; d0 += span) {  // uniform
    const int d = d0 + static_cast<int>(threadIdx.x) * 8;
    const bool in = d < a.D;
    f32x8 x = {};
    if (in) x = *reinterpret_cast<const f32x8*>(a.side + static_cast<size_t>(p) * a.D + d);
    for (int i0 = range.x; i0 < range.y; i0 += kThreads) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      const int q = i < range.y ? a.list[i] : -1;
      const bool own = q >= 0 && a.loc[q] == loc;
      const uint64_t votes = __ballot(own);
      if (lane == 0) s_count[wave] = __popcll(votes);
      __syncthreads();
      int at = 0, n = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        at += w < wave ? s_count[w] : 0;
        n += s_count[w];
      }
      if (own) s_place[at + __popcll(votes & ((uint64_t{1} << lane) - 1))] = q;
      __syncthreads();
      for (int k0 = 0; in && k0 < n; k0 += kAhead) {
        bf16x8 h[kAhead];
        float t[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int k = min(k0 + u, n - 1);
          t[u] = k0 + u < n ? a.term[s_place[k]].target : 0.0f;
          h[u] = load_frag(a.hz + static_cast<size_t>(s_place[k]) * a.Dp + d);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (k0 + u < n)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __builtin_fmaf(t[u], static_cast<float>(h[u][j]), x[j]);
      }
      __syncthreads();  // s_place and s_count are free again
    }
    if (in) {
      uint64_t* out = reinterpret_cast<uint64_t*>(a.dW + static_cast<size_t>(loc) * a.D + d);
      out[0] = pack_bf16(x[0], x[1], x[2], x[3]);
      out[1] = pack_bf16(x[4], x[5], x[6], x[7]);
    }
  }
}

// x + t * w for four consecutive columns of a row of W.
__device__ __forceinline__ f32x4 add_target(f32x4 x, float t, const __bf16* w) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  const bf16x4 v = *reinterpret_cast<const bf16x4*>(w);
  return f32x4{__builtin_fmaf(t, static_cast<float>(v[0]), x[0]),
               __builtin_fmaf(t, static_cast<float>(v[1]), x[1]),
               __builtin_fmaf(t, static_cast<float>(v[2]), x[2]),
               __builtin_fmaf(t, static_cast<float>(v[3]), x[3])};
}

// dh of one slice and one part of its vocabulary rows: straight to dh where
// that is all there is, else into the part's slab (added up from slice to
// slice in fp32).
template <class T>
__global__ __launch_bounds__(T::kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void grad_hidden_kernel(GradArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn_smem[];
  const int n = *a.count;
  const int nb = (n + T::TB - 1) / T::TB, nd = (a.D + T::TA - 1) / T::TA;
  const int splits = a.count[1];
  int btile, at;
  if (!xcd_tile<6>(blockIdx.x, nb, static_cast<int64_t>(nd) * splits, btile, at)) return;
  const int dtile = at % nd, split = at / nd;
  const int a0 = dtile * T::TA, b0 = btile * T::TB;
  const Operand w = {a.W + static_cast<size_t>(a.v0) * a.D, a.D, a.D, a.nv};
  const Operand z = {a.dz, a.ldz, a.Bp, a.ldz};
  const int64_t nk = (a.nv + T::BK - 1) / T::BK;
  const int kt0 = static_cast<int>(nk * split / splits);
  const int kt1 = static_cast<int>(nk * (split + 1) / splits);
  f32x4 acc[T::MR][T::NT];
  if (kt0 < kt1) T::run(w, z, a0, b0, kt0, kt1, acc, dyn_smem);
  else zero_acc(acc);
  const int lane = threadIdx.x & (kWave - 1), li = lane & 15, kb = lane >> 4;
  const int d0 = a0 + T::wave_a() + 4 * kb;
  static_for<T::NT>([&](auto nc) FS_INLINE {
    const int b = b0 + T::wave_b() + 16 * static_cast<int>(nc) + li;
    if (b < n) {
      float* slab = a.slab + (static_cast<size_t>(split) * a.B + b) * a.D + d0;
      __bf16* out = a.dh + static_cast<size_t>(a.slab ? 0 : a.row[b]) * a.D + d0;
      const int loc = a.loc[b];
      const float target = a.term[b].target;
      static_for<T::MR>([&](auto m) FS_INLINE {
        f32x4 x = acc[m][nc];
        if (d0 + 16 * static_cast<int>(m) < a.D) {
          if (a.slab != nullptr) {
            f32x4* p = reinterpret_cast<f32x4*>(slab + 16 * static_cast<int>(m));
            if (!a.first_slice) x += *p;
            *p = x;
          } else {
            if (loc >= 0)
              x = add_target(x, target,
                             a.W + static_cast<size_t>(loc) * a.D + d0 + 16 * static_cast<int>(m));
            *reinterpret_cast<uint64_t*>(out + 16 * static_cast<int>(m)) =
                pack_bf16(x[0], x[1], x[2], x[3]);
          }
        }
      });
    }
  });
}

// The slabs of each row and its target's term, added in a fixed order and
// rounded once.  A block takes one row's 256 columns; its GROUPS groups of 64
// threads split the slabs.  Bound by reading them (4096 rows of 4096, three
// quarters of them with a token: 59 us).
template <int GROUPS>
__global__ __launch_bounds__(GROUPS * kWave) void grad_slabs_kernel(GradArgs a) {
  __shared__ f32x4 s_sum[GROUPS][kWave];
  const int b = blockIdx.x, lane = threadIdx.x & (kWave - 1), group = threadIdx.x / kWave;
  if (b >= a.count[0]) return;
  const int splits = a.count[1];
  const int d = blockIdx.y * (kWave * 4) + lane * 4;
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  if (d < a.D) {
    const float* p = a.slab + static_cast<size_t>(b) * a.D + d;
    const size_t step = static_cast<size_t>(a.B) * a.D;
#pragma unroll 4
    for (int s = group; s < splits; s += GROUPS) x += *reinterpret_cast<const f32x4*>(p + s * step);
  }
  s_sum[group][lane] = x;
  __syncthreads();
  if (group != 0 || d >= a.D) return;
#pragma unroll
  for (int g = 1; g < GROUPS; ++g) x += s_sum[g][lane];
  const int loc = a.loc[b];
  if (loc >= 0) x = add_target(x, a.term[b].target, a.W + static_cast<size_t>(loc) * a.D + d);
  *reinterpret_cast<uint64_t*>(a.dh + static_cast<size_t>(a.row[b]) * a.D + d) =
      pack_bf16(x[0], x[1], x[2], x[3]);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int32_t kMaxGradB = 1 << 22;
constexpr int32_t kMaxGradD = 1 << 20;
// dz of one slice of the vocabulary.
constexpr int64_t kSliceBytes = int64_t{1} << 30;
constexpr int32_t kMaxSlice = 1 << 18;

int32_t target_tiles(int32_t V) {
  return static_cast<int32_t>((static_cast<int64_t>(V) + kTargetTile - 1) / kTargetTile);
}

struct GradPlan {
  int32_t Bp, Dp, slice, splits, TB;
  bool slabs;
  size_t count, slot, row, loc, term, hz, dz, slab, first, list, tile, side, total;
  GradPlan(int32_t B, int32_t D, int32_t V) {
    TB = tile_tokens(B);
    Bp = static_cast<int32_t>(round_up(B, 256));
    Dp = static_cast<int32_t>(round_up(D, 64));
    int64_t s = kSliceBytes / (2 * static_cast<int64_t>(Bp)) / 256 * 256;
    s = s < 256 ? 256 : s > kMaxSlice ? kMaxSlice : s;
    const int64_t whole = static_cast<int64_t>(round_up(V, 256));
    if (s >= whole) {
      s = whole;
    } else {  // equal slices
      const int64_t k = (whole + s - 1) / s;
      s = static_cast<int64_t>(round_up((whole + k - 1) / k, 256));
    }
    slice = static_cast<int32_t>(s);
    // at most as many parts for dh as make four rounds of its tiles, of at least
    // 256 vocabulary rows, with slabs of no more than 512 MiB
    const int64_t tiles = static_cast<int64_t>((B + TB - 1) / TB) * ((D + 255) / 256);
    const int64_t rows = slice < V ? slice : V;
    int64_t p = (1024 + tiles - 1) / tiles;
    p = std::min({p, rows / 256, (int64_t{512} << 20) / (4 * static_cast<int64_t>(B) * D)});
    splits = static_cast<int32_t>(p < 1 ? 1 : p);
    slabs = splits > 1 || slice < V;
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t o = at;
      at += round_up(bytes, 256);
      return o;
    };
    count = take(8);
    slot = take(4ull * B);
    row = take(4ull * Bp);
    loc = take(4ull * Bp);
    term = take(sizeof(RowTerm) * Bp);
    hz = take(2ull * Bp * Dp);
    dz = take(2ull * Bp * slice);
    slab = take(slabs ? 4ull * splits * B * D : 0);
    first = take(4ull * V);
    list = take(4ull * Bp);
    tile = take(sizeof(int2) * target_tiles(V));
    side = take(4ull * Bp * D);
    total = at;
  }
};

unsigned padded_grid(int64_t tiles) { return static_cast<unsigned>((tiles + 7) / 8 * 8); }

// K-major operands take ring slots of 32 k, four or five deep (their rows are as
// long in memory as in slots of 64).
template <int TB> struct HiddenTile;
template <> struct HiddenTile<64> { using T = Tile<kKM, kKC, 8, 1, 2, 4, 4>; };
template <> struct HiddenTile<128> { using T = Tile<kKM, kKC, 4, 2, 4, 4, 3>; };
template <> struct HiddenTile<256> { using T = Tile<kKM, kKC, 2, 4, 8, 4, 4, 32>; };
using WeightsTall = Tile<kKM, kKM, 2, 4, 8, 4, 5, 32>;   // 256 columns x 256 vocabulary rows
using WeightsShort = Tile<kKM, kKM, 1, 4, 8, 4, 3, 32>;  // 128 x 256, 4 waves, two blocks per CU

template <class Kernel>
hipError_t launch_tiles(Kernel kernel, SmemRaised& raised, int64_t tiles, int threads, size_t smem,
                        const GradArgs& a, hipStream_t stream) {
  const hipError_t e = raise_smem(kernel, smem, raised);
  if (e != hipSuccess) return e;
  kernel<<<padded_grid(tiles), threads, smem, stream>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_logits(const GradArgs& a, hipStream_t stream) {
  static SmemRaised raised;
  return launch_tiles(&grad_logits_kernel<T>, raised,
                      static_cast<int64_t>((a.nv + T::TA - 1) / T::TA) *
                          ((a.B + T::TB - 1) / T::TB),
                      T::kThreads, T::kSmemBytes, a, stream);
}

hipError_t launch_logits(const GradArgs& a, hipStream_t stream) {
  switch (logits_tile(a.B, a.nv, true)) {
    case LogitsTile::kTall64: return launch_logits<TallTile<kKC, 64>::T>(a, stream);
    case LogitsTile::kTall128: return launch_logits<TallTile<kKC, 128>::T>(a, stream);
    case LogitsTile::kTall256: return launch_logits<TallTile<kKC, 256>::T>(a, stream);
    case LogitsTile::kShort64: return launch_logits<ShortTile<kKC, 64>::T>(a, stream);
    case LogitsTile::kShort128: return launch_logits<ShortTile<kKC, 128>::T>(a, stream);
    default: return launch_logits<ShortTile<kKC, 256>::T>(a, stream);
  }
}

template <class T>
hipError_t launch_hidden(const GradArgs& a, hipStream_t stream) {
  static SmemRaised raised;
  return launch_tiles(&grad_hidden_kernel<T>, raised,
                      static_cast<int64_t>((a.B + T::TB - 1) / T::TB) *
                          ((a.D + T::TA - 1) / T::TA) * a.max_splits,
                      T::kThreads, T::kSmemBytes, a, stream);
}

hipError_t launch_hidden(const GradArgs& a, hipStream_t stream) {
  return a.hidden_tb == 64    ? launch_hidden<HiddenTile<64>::T>(a, stream)
         : a.hidden_tb == 128 ? launch_hidden<HiddenTile<128>::T>(a, stream)
                              : launch_hidden<HiddenTile<256>::T>(a, stream);
}

template <class T>
hipError_t launch_weights(const GradArgs& a, hipStream_t stream) {
  static SmemRaised raised;
  return launch_tiles(&grad_weights_kernel<T>, raised,
                      static_cast<int64_t>((a.nv + T::TB - 1) / T::TB) *
                          ((a.D + T::TA - 1) / T::TA),
                      T::kThreads, T::kSmemBytes, a, stream);
}

// Two short blocks per CU hide one another's prologue and epilogue, which count
// for few tokens, and make finer rounds of few tiles: 512 tokens on an eighth
// of the vocabulary 137 against 175 us, 2048 tokens 434 against 448 us; with
// many rounds the tall blocks read less (2048 tokens on the whole of it 1793
// against 1860 us, equal at 512).
hipError_t launch_weights(const GradArgs& a, hipStream_t stream) {
  const int64_t tall = static_cast<int64_t>((a.nv + 255) / 256) * ((a.D + 255) / 256);
  return a.B > 512 && tall >= 16 * 256 ? launch_weights<WeightsTall>(a, stream)
                                       : launch_weights<WeightsShort>(a, stream);
}

hipError_t run_grad(GradArgs& a, const GradPlan& p, hipStream_t s) {
  grad_rows_kernel<<<1, kScanThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  grad_gather_kernel<<<a.B + 256, 256, 0, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.dW != nullptr) {
    grad_targets_kernel<<<target_tiles(a.V), kTargetThreads, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  for (int32_t v0 = 0; v0 < a.V; v0 += p.slice) {
    a.v0 = v0;
    a.nv = a.V - v0 < p.slice ? a.V - v0 : p.slice;
    a.first_slice = v0 == 0;
    if (a.B > 0) e = launch_logits(a, s);
    if (e != hipSuccess) return e;
    if (a.dW != nullptr && (e = launch_weights(a, s)) != hipSuccess) return e;
    if (a.dh != nullptr && (e = launch_hidden(a, s)) != hipSuccess) return e;
    if (a.V - v0 <= p.slice) break;  // (v0 + slice may not fit in 32 bits)
  }
  if (a.dW != nullptr && a.B > 0) {
    const int chunks = (a.D + 2047) / 2048;
    grad_target_rows_kernel<<<dim3(a.B, chunks < 64 ? chunks : 64), 256, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.dh != nullptr && p.slabs) {
    const dim3 grid(a.B, (a.D + 4 * kWave - 1) / (4 * kWave));
    // few blocks share out the slabs (4 rows of 1024: the call's dh 35.0 us by
    // sixteen groups, 39.3 by one), many need not (300 rows of 4096: 256, 243)
    if (static_cast<int64_t>(grid.x) * grid.y <= 512)
      grad_slabs_kernel<16><<<grid, 16 * kWave, 0, s>>>(a);
    else grad_slabs_kernel<1><<<grid, kWave, 0, s>>>(a);
    e = hipGetLastError();
  }
  return e;
}

// Whether every launch's grid holds fewer than 2^32 threads: the products' (the
// logits at most one block of 512 per 64 x 64 of them, dW one of 256 per 256 x
// 128 or of 512 per 256 x 256, dh one of 512 per tile and part) and the
// targets', one block per 256 rows of W.  (The others have at most 2^22 + 256
// blocks of 256 threads, or few.)
bool grad_grids_fit(int32_t B, int32_t D, int32_t V, const GradPlan& p, bool dh, bool dW) {
  const int64_t b64 = (B + 63) / 64, slice64 = (static_cast<int64_t>(p.slice) + 63) / 64;
  const int64_t slice256 = (static_cast<int64_t>(p.slice) + 255) / 256;
  const int64_t hidden = static_cast<int64_t>((B + p.TB - 1) / p.TB) * ((D + 255) / 256) * p.splits;
  return grid_fits(slice64 * b64 + 7, 512) &&
         (!dh || grid_fits(hidden + 7, 512)) &&
         (!dW || (grid_fits(slice256 * ((D + 127) / 128) + 7, 256) &&
                  grid_fits(target_tiles(V), kTargetThreads)));
}

bool grad_sizes_ok(int32_t B, int32_t D, int32_t V) {
  return B >= 0 && D >= 8 && D % 8 == 0 && V >= 1 && B <= kMaxGradB && D <= kMaxGradD &&
         V <= kMaxVocab;
}

}  // namespace
}  // namespace fs

extern "C" {

FS_API size_t fs_token_logprobs_backward_workspace_bytes(int32_t B, int32_t D, int32_t V) {
  return fs::grad_sizes_ok(B, D, V) ? fs::GradPlan(B > 0 ? B : 1, D, V).total : 0;
}

FS_API fs_status fs_token_logprobs_backward(const void* h, const void* W, int32_t B, int32_t D,
                                            int32_t V, int32_t vocab_offset,
                                            const float* temperature, const int32_t* token_ids,
                                            const float* logprob, const float* lse,
                                            const float* grad_logprob, void* grad_h, void* grad_W,
                                            void* workspace, size_t workspace_bytes,
                                            void* stream) {
  using namespace fs;
  const char* who = "fs_token_logprobs_backward";
  if (B < 0) return fail(FS_ERR_INVALID_ARG, "%s: B must be >= 0 (got %d)", who, B);
  if (D < 8 || D % 8 != 0)
    return fail(FS_ERR_INVALID_ARG, "%s: D must be a positive multiple of 8 (got %d)", who, D);
  if (V < 1) return fail(FS_ERR_INVALID_ARG, "%s: V must be >= 1 (got %d)", who, V);
  if (vocab_offset < 0 || static_cast<int64_t>(vocab_offset) + V > 2147483647)
    return fail(FS_ERR_INVALID_ARG, "%s: vocab_offset and vocab_offset + V must be in [0, 2^31 - 1]"
                " (got %d, V = %d)", who, vocab_offset, V);
  if (!grad_sizes_ok(B, D, V))
    return fail(FS_ERR_UNSUPPORTED, "%s: B=%d, D=%d, V=%d exceed the %d rows, %d elements or %d "
                "entries a call can take", who, B, D, V, kMaxGradB, kMaxGradD, kMaxVocab);
  if (!grad_h && !grad_W)
    return fail(FS_ERR_INVALID_ARG, "%s: neither grad_h nor grad_W is asked for", who);
  if (!grad_W && B == 0) return FS_OK;
  if (!W || (B > 0 && (!h || !token_ids || !logprob || !lse || !grad_logprob)) || !workspace)
    return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(grad_h, 16) || !aligned(grad_W, 16))
    return fail(FS_ERR_INVALID_ARG, "%s: h, W and their gradients must be 16-byte aligned", who);
  if (!aligned(token_ids, 4) || !aligned(logprob, 4) || !aligned(lse, 4) ||
      !aligned(grad_logprob, 4) || !aligned(temperature, 4))
    return fail(FS_ERR_INVALID_ARG, "%s: per-row arrays must be 4-byte aligned", who);
  if (!aligned(workspace, 256))
    return fail(FS_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  const GradPlan p(B > 0 ? B : 1, D, V);
  if (workspace_bytes < p.total)
    return fail(FS_ERR_WORKSPACE, "%s: workspace of %zu bytes is below the %zu required", who,
                workspace_bytes, p.total);
  if (!grad_grids_fit(B, D, V, p, B > 0 && grad_h, grad_W))
    return fail(FS_ERR_UNSUPPORTED, "%s: B=%d, D=%d, V=%d exceed the launch grid", who, B, D, V);
  if (start_launches()) return injected_failure(who);
  char* ws = static_cast<char*>(workspace);
  GradArgs a;
  a.h = static_cast<const __bf16*>(h);
  a.W = static_cast<const __bf16*>(W);
  a.B = B;
  a.D = D;
  a.V = V;
  a.vocab_offset = vocab_offset;
  a.temperature = temperature;
  a.logprob = logprob;
  a.lse = lse;
  a.grad = grad_logprob;
  a.ids = token_ids;
  a.dh = B > 0 ? static_cast<__bf16*>(grad_h) : nullptr;
  a.dW = static_cast<__bf16*>(grad_W);
  a.count = reinterpret_cast<int32_t*>(ws + p.count);
  a.slot = reinterpret_cast<int32_t*>(ws + p.slot);
  a.row = reinterpret_cast<int32_t*>(ws + p.row);
  a.loc = reinterpret_cast<int32_t*>(ws + p.loc);
  a.term = reinterpret_cast<RowTerm*>(ws + p.term);
  a.hz = reinterpret_cast<__bf16*>(ws + p.hz);
  a.dz = reinterpret_cast<__bf16*>(ws + p.dz);
  a.slab = p.slabs ? reinterpret_cast<float*>(ws + p.slab) : nullptr;
  a.first = reinterpret_cast<int32_t*>(ws + p.first);
  a.list = reinterpret_cast<int32_t*>(ws + p.list);
  a.tile = reinterpret_cast<int2*>(ws + p.tile);
  a.side = reinterpret_cast<float*>(ws + p.side);
  a.Dp = p.Dp;
  a.Bp = p.Bp;
  a.ldz = p.slice;
  a.v0 = a.nv = 0;
  a.max_splits = p.splits;
  a.hidden_tb = p.TB;
  a.first_slice = 1;
  const hipError_t e = run_grad(a, p, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FS_OK : hip_fail(e, "log-probability gradient launch");
}

}  // extern "C"
