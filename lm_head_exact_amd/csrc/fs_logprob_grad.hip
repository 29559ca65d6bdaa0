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
#include <cmath>

#include "fs_grad.hpp"
#include "fs_sampler.hpp"

namespace fs {
namespace {

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
__device__ void gather_row(const GradArgs& a, int b, int at, int n) {
  if (b < a.B) {
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
    if (at >= (n + 255) / 256 * 256) return;
    for (int k = threadIdx.x * 8; k < a.Dp; k += 256 * 8)
      *reinterpret_cast<bf16x8*>(a.hz + static_cast<size_t>(at) * a.Dp + k) = zero_frag();
  }
  if (threadIdx.x != 0) return;
  RowTerm t = {0.0f, 0.0f, 0.0f, 0.0f};
  int loc = -1;
  if (b < a.B) {
    loc = target_row(a.ids[b], a.vocab_offset, a.V);
    if (a.grad != nullptr) {
      const float inv_t = score_inv_t(a.temperature, b);
      const float g = a.grad[b] * inv_t;
      t.inv_t = inv_t;
      t.lse = a.lse[b];
      t.coef = -g;
      t.target = loc >= 0 ? -expm1f(a.logprob[b]) * g : 0.0f;
    }
  }
  a.term[at] = t;
  a.loc[at] = loc;
}

__global__ __launch_bounds__(256) void grad_gather_kernel(GradArgs a) {
  const int b = blockIdx.x, n = *a.count;
  gather_row(a, b, b < a.B ? a.slot[b] : n + (b - a.B), n);
}

// The places that have a target in one tile of 256 vocabulary rows, in order,
// and each row's first one.  Every block reads all targets, twice: B ints
// against the B * 256 * D products of the tile (3 to 6 us).
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

// Rows, gather and targets in one launch for up to kFewRows rows (4 rows on 1000 x
// 256: 40 us a call, 45 by three launches; 513 rows on a shard 379, 383): every block counts the
// ids before its own instead of waiting for one block's scan.  Blocks 0 .. B + 255
// gather, the others (for dW) take a tile of 256 vocabulary rows each.
constexpr int kFewRows = 1024, kFewThreads = 256;

__global__ __launch_bounds__(kFewThreads) void grad_few_rows_kernel(GradArgs a) {
  constexpr int kWaves = kFewThreads / kWave, kEach = kFewRows / kFewThreads;
  __shared__ int32_t s_on[kEach][kWaves], s_hit[kEach][kWaves], s_less[kEach][kWaves];
  __shared__ int32_t s_first[kTargetTile];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, t = threadIdx.x;
  const int gathers = a.B + 256;
  const bool targets = static_cast<int>(blockIdx.x) >= gathers;  // (block-uniform)
  const int b = blockIdx.x, lo = (static_cast<int>(blockIdx.x) - gathers) * kTargetTile;
  if (targets) s_first[t] = 0x7FFFFFFF;
  // id u * 256 + t of every thread
  uint64_t on[kEach], hit[kEach];
  int loc[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int i = u * kFewThreads + t;
    const int32_t id = i < a.B ? a.ids[i] : -1;
    loc[u] = has_token(id) ? target_row(id, a.vocab_offset, a.V) : -1;
    // (targets below the tile, and rows before this block's)
    const uint64_t less =
        __ballot(targets ? loc[u] >= 0 && loc[u] < lo : has_token(id) && i < b);
    on[u] = __ballot(has_token(id));
    hit[u] = __ballot(targets && loc[u] >= lo && loc[u] - lo < kTargetTile);
    if (lane == 0) {
      s_on[u][wave] = __popcll(on[u]);
      s_hit[u][wave] = __popcll(hit[u]);
      s_less[u][wave] = __popcll(less);
    }
  }
  __syncthreads();
  int n = 0, before = 0;
#pragma unroll
  for (int u = 0; u < kEach; ++u)
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      n += s_on[u][w];
      before += s_less[u][w];
    }
  if (targets) {
    const uint64_t below = (uint64_t{1} << lane) - 1;
    int place = 0, at = before;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      int my_place = place, my_at = at;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        my_place += w < wave ? s_on[u][w] : 0;
        my_at += w < wave ? s_hit[u][w] : 0;
        place += s_on[u][w];
        at += s_hit[u][w];
      }
      if (hit[u] >> lane & 1) {
        const int p = my_place + __popcll(on[u] & below);
        a.list[my_at + __popcll(hit[u] & below)] = p;
        atomicMin(&s_first[loc[u] - lo], p);  // (the minimum does not depend on the order)
      }
    }
    __syncthreads();
    const int v = lo + t;
    if (v < a.V) a.first[v] = s_first[t] == 0x7FFFFFFF ? -1 : s_first[t];
    if (t == 0) a.tile[lo / kTargetTile] = int2{before, at};
    return;
  }
  if (b == gathers - 1) {  // (a block with next to nothing to gather)
    uint64_t best = ~0ull;
    for (int parts = t + 1; parts <= a.max_splits; parts += kFewThreads)
      best = min(best, hidden_cost(a, n, parts) << 12 | parts);
    __shared__ unsigned long long s_best;
    if (t == 0) s_best = ~0ull;
    __syncthreads();
    atomicMin(&s_best, static_cast<unsigned long long>(best));
    __syncthreads();
    if (t == 0) {
      a.count[0] = n;
      a.count[1] = static_cast<int32_t>(s_best & 4095);
    }
  }
  const bool mine = b < a.B && has_token(a.ids[min(b, a.B - 1)]);
  if (b < a.B && t == 0) a.slot[b] = mine ? before : -1;
  if (mine && t == 0) a.row[before] = b;
  gather_row(a, b, b < a.B ? (mine ? before : -1) : n + (b - a.B), n);
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
  const bool whole = a0 + T::TA <= a.nv, full = b0 + T::TB <= n;
  RowTerm term[T::NT];
  int loc[T::NT];
  // places behind the last one: 0, whatever their hidden states of 0 made of W's infinite
  // entries (dW reads them where it fills a k tile)
  bool fill[T::NT];
  static_for<T::NT>([&](auto nc) FS_INLINE {
    const int b = b0 + T::wave_b() + 16 * static_cast<int>(nc) + li;
    term[nc] = a.term[b];
    loc[nc] = a.loc[b] - a.v0;
    fill[nc] = !full && b >= n;
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
          // (the difference first, rounded once: it holds for logits of any size)
          const float x = __builtin_fmaf(z[r], term[n].inv_t, -term[n].lse);
          d[r] = __builtin_amdgcn_exp2f(x * 1.44269504088896341f) * term[n].coef;
          d[r] = v == loc[n] || (!whole && v >= a.nv) || fill[n] ? 0.0f : d[r];
        });
        return pack_bf16(d[0], d[1], d[2], d[3]);
      },
      [&](int r) FS_INLINE { return out + static_cast<size_t>(r) * a.ldz; },
      [&](int, int) FS_INLINE { return true; });
}

// dW of one slice: rows v of W, columns d, summed over the rows with a target.  SPLIT:
// over one part of them, into the part's slab.  NTS: stores that pass the caches (a kernel
// of its own: the compiler joins the last stores of two branches, and the joined one has
// lost the hint).
template <class T, bool SPLIT, bool NTS>
__global__ __launch_bounds__(T::kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void grad_weights_kernel(GradArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn_smem[];
  const int n = *a.count;
  const int nd = (a.D + T::TA - 1) / T::TA;
  int tile, at;
  if (!xcd_tile<4>(blockIdx.x, (a.nv + T::TB - 1) / T::TB, SPLIT ? nd * a.w_splits : nd, tile, at))
    return;
  const int a0 = (SPLIT ? at % nd : at) * T::TA, b0 = tile * T::TB;
  const Operand h = {a.hz, a.Dp, a.D, a.Bp};
  const Operand z = {a.dz, a.ldz, a.ldz, a.Bp};
  const int nk = (n + T::BK - 1) / T::BK;
  const int part = SPLIT ? at / nd : 0;
  const int kt0 = SPLIT ? static_cast<int>(static_cast<int64_t>(nk) * part / a.w_splits) : 0;
  const int kt1 = SPLIT ? static_cast<int>(static_cast<int64_t>(nk) * (part + 1) / a.w_splits) : nk;
  f32x4 acc[T::MR][T::NT];
  if (kt0 < kt1) T::run(h, z, a0, b0, kt0, kt1, acc, dyn_smem);
  else zero_acc(acc);
  const int lane = threadIdx.x & (kWave - 1), li = lane & 15, kb = lane >> 4;
  const int d0 = a0 + T::wave_a() + 4 * kb;
  if constexpr (SPLIT) {
    static_for<T::NT>([&](auto n) FS_INLINE {
      const int v = b0 + T::wave_b() + 16 * static_cast<int>(n) + li;
      if (v < a.nv) {
        float* slab = a.wslab + (static_cast<size_t>(part) * a.V + v) * a.D + d0;
        static_for<T::MR>([&](auto m) FS_INLINE {
          if (d0 + 16 * static_cast<int>(m) < a.D)
            *reinterpret_cast<f32x4*>(slab + 16 * static_cast<int>(m)) = acc[m][n];
        });
      }
    });
    return;
  }
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
  T::template store_rows<NTS>(
      dyn_smem,
      [&](auto m, auto n) FS_INLINE {
        const f32x4 x = acc[m][n];
        return pack_bf16(x[0], x[1], x[2], x[3]);
      },
      [&](int r) FS_INLINE { return out + static_cast<size_t>(r) * a.D; },
      [&](int r, int c) FS_INLINE { return v0 + r < a.nv && c0 + c < a.D; });
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

// The targets' rows of dW: what the product left on the side plus each target's
// own term, in the order of the places, rounded once.  One block per place (and part
// y of ny of its columns), which has something to do where it is its target's first;
// a thread takes eight columns.  The block looks through its tile's targets THREADS
// at a time for those that are its own, then adds these.
template <int THREADS>
__device__ void finish_target_row(const GradArgs& a, int p, int y, int ny) {
  constexpr int kWaves = THREADS / kWave, kAhead = 8;
  __shared__ int32_t s_place[THREADS + kAhead];
  __shared__ int32_t s_count[kWaves];
  if (p >= a.count[0]) return;
  const int loc = a.loc[p];
  if (loc < 0 || a.first[loc] != p) return;
  const int2 range = a.tile[loc / kTargetTile];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  const int span = ny * THREADS * 8;
  for (int d0 = y * THREADS * 8; d0 < a.D; d0 += span) {  // uniform
    const int d = d0 + static_cast<int>(threadIdx.x) * 8;
    const bool in = d < a.D;
    f32x8 x = {};
    if (in && a.w_splits == 1)
      x = *reinterpret_cast<const f32x8*>(a.side + static_cast<size_t>(p) * a.D + d);
    for (int s = 0; in && a.w_splits > 1 && s < a.w_splits; ++s)
      x += *reinterpret_cast<const f32x8*>(
          a.wslab + (static_cast<size_t>(s) * a.V + loc) * a.D + d);
    for (int i0 = range.x; i0 < range.y; i0 += THREADS) {
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

// The rows of dW that are no target, from their parts: added in order, rounded once.
__global__ __launch_bounds__(256) void grad_weight_slabs_kernel(GradArgs a) {
  const int quads = a.D / 4;
  const int64_t total = static_cast<int64_t>(a.V) * quads;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += 256ll * gridDim.x) {
    if (a.first[i / quads] >= 0) continue;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.w_splits; ++s)
      x += *reinterpret_cast<const f32x4*>(a.wslab + (s * total + i) * 4);
    *reinterpret_cast<uint64_t*>(a.dW + i * 4) = pack_bf16(x[0], x[1], x[2], x[3]);
  }
}

// The slabs of columns d .. d + 3 of place b and its target's term, added in a fixed
// order and rounded once.
template <int GROUPS>
__device__ f32x4 sum_slabs(const GradArgs& a, int b, int d, int group) {
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  const int splits = a.count[1];
  const float* p = a.slab + static_cast<size_t>(b) * a.D + d;
  const size_t step = static_cast<size_t>(a.B) * a.D;
#pragma unroll 4
  for (int s = group; s < splits; s += GROUPS) x += *reinterpret_cast<const f32x4*>(p + s * step);
  return x;
}
__device__ __forceinline__ void finish_hidden(const GradArgs& a, int b, int d, f32x4 x) {
  const int loc = a.loc[b];
  if (loc >= 0) x = add_target(x, a.term[b].target, a.W + static_cast<size_t>(loc) * a.D + d);
  *reinterpret_cast<uint64_t*>(a.dh + static_cast<size_t>(a.row[b]) * a.D + d) =
      pack_bf16(x[0], x[1], x[2], x[3]);
}

// What is left of both gradients, side by side in one launch: blocks (place, y) make
// the targets' rows of dW for y below `chunks`, and above that add up dh's slabs, a
// wave or GROUPS waves for 256 columns.  Bound by reading the slabs (4096 rows of 4096,
// three quarters of them with a token: 73 us; 25 and 59 one after the other; 513 rows on
// a shard 16, 9 and 12; 4 rows on 1000 x 256 37.0 us a call, 39.6 by two launches).  GROUPS 16
// where the blocks are few (4 rows of 1024: the call's dh 35.0 us by sixteen groups,
// 39.3 by one; 300 rows of 4096: 256, 243).
template <int GROUPS>
__global__ __launch_bounds__(GROUPS == 1 ? 256 : GROUPS * kWave) void grad_finish_kernel(
    GradArgs a, int32_t chunks) {
  constexpr int kThreads = GROUPS == 1 ? 256 : GROUPS * kWave;
  const int b = blockIdx.x, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  if (static_cast<int>(blockIdx.y) < chunks) {  // (block-uniform)
    finish_target_row<kThreads>(a, b, blockIdx.y, chunks);
    return;
  }
  if (b >= a.count[0]) return;
  const int at = static_cast<int>(blockIdx.y) - chunks;
  if constexpr (GROUPS == 1) {
    const int d = (at * (kThreads / kWave) + wave) * (kWave * 4) + lane * 4;
    if (d < a.D) finish_hidden(a, b, d, sum_slabs<1>(a, b, d, 0));
  } else {
    __shared__ f32x4 s_sum[GROUPS][kWave];
    const int d = at * (kWave * 4) + lane * 4;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (d < a.D) x = sum_slabs<GROUPS>(a, b, d, wave);
    s_sum[wave][lane] = x;
    __syncthreads();
    if (wave != 0 || d >= a.D) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) x += s_sum[g][lane];
    finish_hidden(a, b, d, x);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
unsigned padded_grid(int64_t tiles) { return static_cast<unsigned>((tiles + 7) / 8 * 8); }

// K-major operands take ring slots of 32 k, four or five deep (their rows are as
// long in memory as in slots of 64).
template <int TB> struct HiddenTile;
template <> struct HiddenTile<64> { using T = Tile<kKM, kKC, 8, 1, 2, 4, 4>; };
template <> struct HiddenTile<128> { using T = Tile<kKM, kKC, 4, 2, 4, 4, 3>; };
template <> struct HiddenTile<256> { using T = Tile<kKM, kKC, 2, 4, 8, 4, 4, 32>; };
using WeightsTall = Tile<kKM, kKM, 2, 4, 8, 4, 5, 32>;   // 256 columns x 256 vocabulary rows
using WeightsShort = Tile<kKM, kKM, 1, 4, 8, 4, 3, 32>;  // 128 x 256, 4 waves, two blocks per CU
static_assert(WeightsTall::BK == kGradPlaces && WeightsShort::BK == kGradPlaces, "places of a k tile");

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

template <class T, bool SPLIT, bool NTS>
hipError_t launch_weights(const GradArgs& a, hipStream_t stream) {
  static SmemRaised raised;
  return launch_tiles(&grad_weights_kernel<T, SPLIT, NTS>, raised,
                      static_cast<int64_t>((a.nv + T::TB - 1) / T::TB) *
                          ((a.D + T::TA - 1) / T::TA) * (SPLIT ? a.w_splits : 1),
                      T::kThreads, T::kSmemBytes, a, stream);
}

// Two short blocks per CU hide one another's prologue and epilogue, which count
// for few tokens, and make finer rounds of few tiles: 512 tokens on an eighth
// of the vocabulary 137 against 175 us, 2048 tokens 434 against 448 us; with
// many rounds the tall blocks read less (2048 tokens on the whole of it 1793
// against 1860 us, equal at 512).
template <bool NTS>
hipError_t launch_weights(const GradArgs& a, hipStream_t stream) {
  const int64_t tall = static_cast<int64_t>((a.nv + 255) / 256) * ((a.D + 255) / 256);
  return a.B > 512 && tall >= 16 * 256 ? launch_weights<WeightsTall, false, NTS>(a, stream)
                                       : launch_weights<WeightsShort, false, NTS>(a, stream);
}

// Past the caches where every row starts a line.  Else lines are filled by two tiles, and
// few rows' dW is faster through the caches (a call, through and past them: 14 rows on
// 97002 x 2616 305 and 340 us, 64 rows 321 and 340, 100 rows on 32000 x 2056 91 and 97).  A
// longer product gains more from what a large dW would push out of them meanwhile (dW and
// dh: 130 rows on 97002 x 2616 563 and 549, 300 rows 819 and 788; 300 rows on 32000 x 2056
// 217 and 210; 1025 rows on 50000 x 1016 432 and 398; on 32000 x 1000 512 rows 135 and 137,
// 2048 rows 412 and 393).
bool weights_pass_caches(const GradArgs& a) {
  return a.D % 64 == 0 ||
         (a.B > 64 && a.B * static_cast<int64_t>(a.V) > (int64_t{1} << 34) / a.D);
}

hipError_t launch_weights(const GradArgs& a, hipStream_t stream) {
  if (a.w_splits > 1) return launch_weights<WeightsShort, true, false>(a, stream);
  return weights_pass_caches(a) ? launch_weights<true>(a, stream) : launch_weights<false>(a, stream);
}

hipError_t run_grad(GradArgs& a, const GradPlan& p, hipStream_t s) {
  hipError_t e = launch_grad_rows(a, s);
  if (e != hipSuccess) return e;
  for (int32_t v0 = 0; v0 < a.V; v0 += p.slice) {
    a.v0 = v0;
    a.nv = a.V - v0 < p.slice ? a.V - v0 : p.slice;
    a.first_slice = v0 == 0;
    if (a.B > 0) e = launch_logits(a, s);
    if (e != hipSuccess) return e;
    if ((e = launch_grad_products(a, s)) != hipSuccess) return e;
    if (a.V - v0 <= p.slice) break;  // (v0 + slice may not fit in 32 bits)
  }
  return launch_grad_finish(a, s);
}

}  // namespace

void grad_workspace(GradArgs& a, const GradPlan& p, char* ws) {
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
  a.wslab = reinterpret_cast<float*>(ws + p.wslab);
  a.w_splits = p.w_splits;
  a.Dp = p.Dp;
  a.Bp = p.Bp;
  a.ldz = p.slice;
  a.v0 = a.nv = 0;
  a.max_splits = p.splits;
  a.hidden_tb = p.TB;
  a.first_slice = 1;
}

hipError_t launch_grad_rows(const GradArgs& a, hipStream_t s) {
  if (a.B <= kFewRows) {
    const int64_t blocks = a.B + 256ll + (a.dW != nullptr ? target_tiles(a.V) : 0);
    grad_few_rows_kernel<<<static_cast<unsigned>(blocks), kFewThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  grad_rows_kernel<<<1, kScanThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  grad_gather_kernel<<<a.B + 256, 256, 0, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess || a.dW == nullptr) return e;
  grad_targets_kernel<<<target_tiles(a.V), kTargetThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_products(const GradArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.dW != nullptr) e = launch_weights(a, s);
  if (e == hipSuccess && a.dh != nullptr) e = launch_hidden(a, s);
  return e;
}

hipError_t launch_grad_finish(const GradArgs& a, hipStream_t s) {
  const bool rows = a.dW != nullptr && a.B > 0, slabs = a.dh != nullptr && a.slab != nullptr;
  if (!rows && !slabs) return hipSuccess;
  if (rows && a.w_splits > 1) {
    const int64_t blocks = (static_cast<int64_t>(a.V) * a.D / 4 + 255) / 256;
    grad_weight_slabs_kernel<<<static_cast<unsigned>(blocks < 8192 ? blocks : 8192), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int units = (a.D + 4 * kWave - 1) / (4 * kWave);
  const bool few = slabs && static_cast<int64_t>(a.B) * units <= 512;
  const int threads = few ? 16 * kWave : 256;
  const int parts = (a.D + 8 * threads - 1) / (8 * threads);
  const int chunks = !rows ? 0 : parts < 64 ? parts : 64;
  const dim3 grid(a.B, chunks + (!slabs ? 0 : few ? units : (units + 3) / 4));
  if (few) grad_finish_kernel<16><<<grid, threads, 0, s>>>(a, chunks);
  else grad_finish_kernel<1><<<grid, threads, 0, s>>>(a, chunks);
  return hipGetLastError();
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
  grad_workspace(a, p, ws);
  const hipError_t e = run_grad(a, p, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FS_OK : hip_fail(e, "log-probability gradient launch");
}

}  // extern "C"
