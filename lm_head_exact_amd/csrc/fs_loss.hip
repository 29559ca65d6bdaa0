// fs_loss.hip -- losses on token log-probabilities, with their gradients: the
// clipped policy loss with a KL penalty, and the preference loss of paired
// answers.
//
// Both read a packed batch of sequences (tokens [cu[s], cu[s+1]) of flat
// arrays).  Every token's gradient carries a count over the whole batch
// (tokens, sequences or pairs that count), so a batch takes two passes:
//   policy      counts (the mask alone), then all terms, gradients and sums,
//               which one block adds up for the statistics
//   preference  sums of the answers, then the gradients (one value per
//               answer), for which each block settles its own answers' pair
// A small batch takes both passes in one block with its sums in LDS.
// Every sum is taken in fp64 and in a fixed order (strided lanes, shuffles,
// then parts or blocks in order), so equal calls give equal bits.  A token is
// 13 to 21 bytes and a few dozen operations: launches and memory latency bound
// a batch of any usual size, not bandwidth (8 answers of 100 tokens: 9.5 us
// policy, 8.3 preference, in one block; 512 answers of 1900 tokens: 4 us
// counts, 15 terms, 4 sums, and 7 sums, 7 gradients).
#include <cmath>

#include "fs_host.hpp"
#include "fs_internal.hpp"
#include "fs_tokens.hpp"

namespace fs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaveSize = 64;
constexpr int kOneBlockThreads = 1024;

// The batches one block handles by itself: what it takes longer than the passes
// over the device is below the two launches (2 to 3 us each on the host) that
// it saves.  Policy, preference on the device: 8 sequences of 500 tokens 11.5
// and 9.4 us against 14.9 and 8.3; 4 of 2000, 14.5 and 11.7 against 12.5 and
// 8.0; 128 of 32, 28.7 and 23.0 against 11.2 and 6.9.
constexpr int32_t kOneBlockTokens = 4096;
constexpr int32_t kOneBlockSequences = 32;
// their parts: sequences with several have kOneBlockThreads / 64 or a few more
constexpr int32_t kOneBlockItems = kOneBlockSequences + kOneBlockThreads / kWaveSize;
// Parts whose sums every block of the second pass adds up by itself; beyond
// them one block does between the passes, in a launch of its own (2048 parts:
// 14.4 us within the blocks, 14.5 between them; 4096: 18.0 and 16.7, which a
// call's host side hides; 8192: 30.9 and 21.0).
constexpr int64_t kInBlockItems = 4096;
// A part takes a block where the parts are few and their mean length is at
// least this, else a wave: 512 sequences of 1024 tokens 14.9 us by blocks, 20.9
// by waves; of 256, 12.7 and 13.4; of 64, 12.3 and 11.6.  Many parts fill the
// device by waves: 2048 of 512 tokens 23.4 us by blocks, 18.9 by waves.
constexpr int64_t kBlockTeamTokens = 512;
constexpr int64_t kBlockTeamItems = 2048;
// The most parts of a sequence.
constexpr int32_t kMaxParts = 256;

struct SeqArgs {
  const int32_t* cu;     // [S + 1]
  const uint8_t* mask;   // [T] or null
  int32_t S, T;
  int32_t parts;         // parts per sequence
  int32_t zero_outside;  // gradients outside every sequence are set to 0
};

// Tokens [a, b) of part y of sequence s.  Offsets come from device memory, so
// they are clamped to the arrays: a wrong offset gives wrong sums, never an
// access outside [0, T).
__device__ __forceinline__ void part_range(const SeqArgs& q, int s, int y, int& a, int& b) {
  const int lo = min(max(q.cu[s], 0), q.T);
  const int hi = min(max(q.cu[s + 1], lo), q.T);
  const int64_t len = hi - lo;
  a = lo + static_cast<int>(len * y / q.parts);
  b = lo + static_cast<int>(len * (y + 1) / q.parts);
}

// Gradients before the first and behind the last sequence, this thread's share
// of `threads`.
__device__ __forceinline__ void outside(const SeqArgs& q, float* grad, int64_t thread,
                                        int64_t threads) {
  if (!q.zero_outside) return;
  const int first = q.S > 0 ? min(max(q.cu[0], 0), q.T) : q.T;
  const int end = q.S > 0 ? min(max(q.cu[q.S], first), q.T) : q.T;
  for (int64_t t = thread; t < first; t += threads) grad[t] = 0.0f;
  for (int64_t t = end + thread; t < q.T; t += threads) grad[t] = 0.0f;
}

__device__ __forceinline__ bool counts(const SeqArgs& q, int t) {
  return q.mask == nullptr || q.mask[t] != 0;
}

struct Sum4 {
  double x, y;
  int32_t n, k;
  __device__ __forceinline__ void zero() { x = y = 0.0; n = k = 0; }
  __device__ __forceinline__ void add(const Sum4& o) {
    x += o.x;
    y += o.y;
    n += o.n;
    k += o.k;
  }
  __device__ __forceinline__ void wave_sum() {
#pragma unroll
    for (int m = kWaveSize / 2; m >= 1; m >>= 1) {
      Sum4 o;
      o.x = __shfl_xor(x, m, kWaveSize);
      o.y = __shfl_xor(y, m, kWaveSize);
      o.n = __shfl_xor(n, m, kWaveSize);
      o.k = __shfl_xor(k, m, kWaveSize);
      add(o);
    }
  }
};

// Sum over the block, on every thread (waves in order).
template <int THREADS>
__device__ __forceinline__ Sum4 block_sum(Sum4 v) {
  __shared__ Sum4 s[THREADS / kWaveSize];
  v.wave_sum();
  if ((threadIdx.x & (kWaveSize - 1)) == 0) s[threadIdx.x / kWaveSize] = v;
  __syncthreads();
  Sum4 r = s[0];
#pragma unroll
  for (int w = 1; w < THREADS / kWaveSize; ++w) r.add(s[w]);
  __syncthreads();
  return r;
}

// Two counts over the block, on every thread.
template <int THREADS>
__device__ __forceinline__ int2 block_count(int x, int y) {
  Sum4 v;
  v.zero();
  v.n = x;
  v.k = y;
  v = block_sum<THREADS>(v);
  return int2{v.n, v.k};
}

// Team and item (part of a sequence) of a thread: TEAM threads per item.
template <int TEAM>
__device__ __forceinline__ int64_t item_of_thread() {
  return static_cast<int64_t>(blockIdx.x) * (kThreads / TEAM) + threadIdx.x / TEAM;
}

// ---------------------------------------------------------------------------
// Policy loss.
// ---------------------------------------------------------------------------
struct PolicyArgs {
  SeqArgs q;
  const float *lp, *old, *ref, *adv;  // ref may be null
  int32_t adv_per_token, kl_kind, seq_mean;
  // borders of the log-ratio d = lp - old, from the host in fp64: a token is
  // clipped above at d > log(1 + clip_high), below at d < log(1 - clip_low)
  // and capped (negative advantages) at d > log(dual_clip).  Deciding on the
  // exact difference of the inputs, rather than on a rounded ratio, makes
  // the decision the definition's for every input.
  double log_high, log_low, log_cap;
  float high, low, cap;
  double kl_coef, grad_scale;
  int32_t* count;   // [S * parts]
  int2* totals;     // tokens, sequences that count; read if have_totals
  int32_t have_totals;
  Sum4* part;       // [blocks]: weighted sums of the blocks
  float* stats;     // [4]
  float* grad;      // [T]
};

struct PolicyToken {
  float lp, old, ref, adv;
  bool on;
};

struct TokenTerms {
  float surr, kl, g;
  bool clipped;
};

__device__ __forceinline__ PolicyToken load_policy(const PolicyArgs& a, int t, float As) {
  PolicyToken k;
  k.on = counts(a.q, t);
  k.lp = a.lp[t];
  k.old = a.old[t];
  k.ref = a.ref != nullptr ? a.ref[t] : 0.0f;
  k.adv = a.adv_per_token ? a.adv[t] : As;
  return k;
}

// em = e^q - 1 and e^q - q - 1.  The latter cancels to q^2 / 2 near 0: there its
// series (the first term left out is below 2^-25 of it for |q| < 1/2), and em is
// the sum of it and q, which does not cancel; elsewhere em is taken from e^q, as
// the excess would have lost it to q (q = -1e8: em is -1).  Both have their
// limits at infinite q.
__device__ __forceinline__ float exp_excess(float q, float& em) {
  float p = 1.0f / 3628800.0f;
  p = __builtin_fmaf(p, q, 1.0f / 362880.0f);
  p = __builtin_fmaf(p, q, 1.0f / 40320.0f);
  p = __builtin_fmaf(p, q, 1.0f / 5040.0f);
  p = __builtin_fmaf(p, q, 1.0f / 720.0f);
  p = __builtin_fmaf(p, q, 1.0f / 120.0f);
  p = __builtin_fmaf(p, q, 1.0f / 24.0f);
  p = __builtin_fmaf(p, q, 1.0f / 6.0f);
  p = __builtin_fmaf(p, q, 0.5f);
  const bool near = fabsf(q) < 0.5f;
  const float series = p * q * q, far = expf(q) - 1.0f;
  em = near ? q + series : far;
  return near ? series : far == INFINITY ? far : far - q;
}

__device__ __forceinline__ TokenTerms policy_token(const PolicyArgs& a, const PolicyToken& k) {
  TokenTerms o;
  const float A = k.adv;
  const double d = static_cast<double>(k.lp) - static_cast<double>(k.old);
  const float r = expf(static_cast<float>(d));
  const bool over = d > a.log_high, under = d < a.log_low;
  const bool cap = A < 0.0f && d > a.log_cap;
  o.clipped = (A > 0.0f && over) || (A < 0.0f && under) || cap;
  const float rc = cap ? a.cap : over ? a.high : under ? a.low : r;
  // an advantage of zero leaves nothing, whatever the ratio
  const float live = A == 0.0f ? 0.0f : -(r * A);
  o.surr = o.clipped ? -(rc * A) : live;
  o.g = o.clipped ? 0.0f : live;
  o.kl = 0.0f;
  if (a.ref != nullptr) {
    const float q = static_cast<float>(static_cast<double>(k.ref) - static_cast<double>(k.lp));
    float gk;
    if (a.kl_kind == FS_KL_K1) {
      o.kl = -q;
      gk = 1.0f;
    } else if (a.kl_kind == FS_KL_K2) {
      o.kl = 0.5f * q * q;
      gk = -q;
    } else {
      o.kl = exp_excess(q, gk);
      gk = -gk;
    }
    // without a coefficient the term is only reported: it may be infinite or NaN
    if (a.kl_coef != 0.0) o.g += static_cast<float>(a.kl_coef) * gk;
  }
  return o;
}

// Tokens that count in part y of sequence s, this lane's share.
__device__ __forceinline__ int count_part(const SeqArgs& q, int s, int y, int lane, int team) {
  int t0, t1, n = 0;
  part_range(q, s, y, t0, t1);
  if (q.mask == nullptr) return lane == 0 ? t1 - t0 : 0;
  each_token(t0, t1, lane, team, [&](int t) { return q.mask[t]; },
             [&](int, uint8_t m) { n += m != 0; });
  return n;
}

__device__ __forceinline__ int wave_count(int n) {
#pragma unroll
  for (int m = kWaveSize / 2; m >= 1; m >>= 1) n += __shfl_xor(n, m, kWaveSize);
  return n;
}

// Gradients of part y of sequence s (weight w per token) and this lane's share
// of its sums.  The weight stays fp64: a gradient is rounded with its product
// alone, and a weight beyond fp32 leaves tokens that do not count at 0.
__device__ __forceinline__ Sum4 policy_part(const PolicyArgs& a, int s, int y, double w, int lane,
                                            int team) {
  int t0, t1;
  part_range(a.q, s, y, t0, t1);
  Sum4 v;
  v.zero();
  const float As = a.adv_per_token ? 0.0f : a.adv[s];
  each_token(t0, t1, lane, team, [&](int t) { return load_policy(a, t, As); },
             [&](int t, const PolicyToken& k) {
               float g = 0.0f;
               if (k.on) {  // masked tokens may hold anything
                 const TokenTerms o = policy_token(a, k);
                 v.x += static_cast<double>(o.surr);
                 v.y += static_cast<double>(o.kl);
                 v.n += 1;
                 v.k += o.clipped ? 1 : 0;
                 g = static_cast<float>(o.g * w);
               }
               a.grad[t] = g;
             });
  return v;
}

// Weight of a token of a sequence with n tokens that count.
__device__ __forceinline__ double policy_weight(const PolicyArgs& a, int2 totals, int n) {
  if (a.seq_mean) return 1.0 / (static_cast<double>(max(n, 1)) * max(totals.y, 1));
  return 1.0 / max(totals.x, 1);
}

// `all`: weighted sums of the surrogate and the KL term, tokens, clipped ones.
__device__ __forceinline__ void write_policy_stats(const PolicyArgs& a, const Sum4& all) {
  a.stats[0] = static_cast<float>(a.kl_coef != 0.0 ? all.x + a.kl_coef * all.y : all.x);
  a.stats[1] = static_cast<float>(all.x);
  a.stats[2] = static_cast<float>(all.y);
  a.stats[3] = static_cast<float>(static_cast<double>(all.k) / max(all.n, 1));
}

template <int TEAM>
__global__ __launch_bounds__(kThreads) void policy_counts_kernel(PolicyArgs a) {
  const int64_t item = item_of_thread<TEAM>();
  const bool in = item < static_cast<int64_t>(a.q.S) * a.q.parts;
  const int s = static_cast<int>(item / a.q.parts), y = static_cast<int>(item % a.q.parts);
  int n = in ? wave_count(count_part(a.q, s, y, threadIdx.x % TEAM, TEAM)) : 0;
  if constexpr (TEAM > kWaveSize) n = block_count<kThreads>(threadIdx.x % kWaveSize == 0 ? n : 0, 0).x;
  if (in && threadIdx.x % TEAM == 0) a.count[item] = n;
}

// Tokens and sequences that count, over a block of THREADS threads.
template <int THREADS>
__device__ __forceinline__ int2 policy_totals(const PolicyArgs& a) {
  int tokens = 0, filled = 0;
  for (int s = threadIdx.x; s < a.q.S; s += THREADS) {
    int n = 0;
#pragma unroll 8
    for (int y = 0; y < a.q.parts; ++y) n += a.count[static_cast<size_t>(s) * a.q.parts + y];
    tokens += n;
    filled += n > 0;
  }
  return block_count<THREADS>(tokens, filled);
}

__global__ __launch_bounds__(kOneBlockThreads) void policy_totals_kernel(PolicyArgs a) {
  const int2 t = policy_totals<kOneBlockThreads>(a);
  if (threadIdx.x == 0) *a.totals = t;
}

template <int TEAM>
__global__ __launch_bounds__(kThreads) void policy_kernel(PolicyArgs a) {
  outside(a.q, a.grad, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x,
          static_cast<int64_t>(gridDim.x) * kThreads);
  const int2 totals = a.have_totals ? *a.totals : policy_totals<kThreads>(a);
  const int64_t item = item_of_thread<TEAM>();
  Sum4 v;
  v.zero();
  if (item < static_cast<int64_t>(a.q.S) * a.q.parts) {
    const int s = static_cast<int>(item / a.q.parts), y = static_cast<int>(item % a.q.parts);
    int n = 0;
#pragma unroll 8
    for (int i = 0; i < a.q.parts; ++i) n += a.count[static_cast<size_t>(s) * a.q.parts + i];
    const double w = policy_weight(a, totals, n);
    v = policy_part(a, s, y, w * a.grad_scale, threadIdx.x % TEAM, TEAM);
    v.x *= w;
    v.y *= w;
  }
  v = block_sum<kThreads>(v);
  if (threadIdx.x == 0) a.part[blockIdx.x] = v;
}

// A launch of its own: letting the last block of the pass before add up the
// blocks' sums would cost each of them a write-back of its L2 to be seen
// (27 us for the pass over a million tokens, against 15 and 4).
__global__ __launch_bounds__(kOneBlockThreads) void policy_stats_kernel(PolicyArgs a,
                                                                        unsigned blocks) {
  Sum4 all;
  all.zero();
  for (unsigned i = threadIdx.x; i < blocks; i += kOneBlockThreads) all.add(a.part[i]);
  all = block_sum<kOneBlockThreads>(all);
  if (threadIdx.x == 0) write_policy_stats(a, all);
}

// Both passes in one block: a wave per part, gradients first without their
// weight, then scaled by the threads that wrote them.
__global__ __launch_bounds__(kOneBlockThreads) void policy_one_block_kernel(PolicyArgs a) {
  __shared__ Sum4 part[kOneBlockItems];
  __shared__ double weight[kOneBlockSequences];
  outside(a.q, a.grad, threadIdx.x, kOneBlockThreads);
  constexpr int kWaves = kOneBlockThreads / kWaveSize;
  const int wave = threadIdx.x / kWaveSize, lane = threadIdx.x % kWaveSize;
  const int Y = a.q.parts, S = a.q.S, items = S * Y;
  for (int i = wave; i < items; i += kWaves) {
    Sum4 v = policy_part(a, i / Y, i % Y, 1.0, lane, kWaveSize);
    v.wave_sum();
    if (lane == 0) part[i] = v;
  }
  __syncthreads();
  Sum4 one;  // S <= threads: a sequence each
  one.zero();
  const int s = threadIdx.x;
  if (s < S)
    for (int y = 0; y < Y; ++y) one.add(part[s * Y + y]);
  const int2 totals = block_count<kOneBlockThreads>(one.n, one.n > 0);
  const double w = policy_weight(a, totals, one.n);
  if (s < S) weight[s] = w * a.grad_scale;
  one.x *= w;
  one.y *= w;
  const Sum4 all = block_sum<kOneBlockThreads>(one);
  if (threadIdx.x == 0) write_policy_stats(a, all);
  for (int i = wave; i < items; i += kWaves) {
    int t0, t1;
    part_range(a.q, i / Y, i % Y, t0, t1);
    const double c = weight[i / Y];
    // zero stays zero: a token that does not count has no gradient
    each_token(t0, t1, lane, kWaveSize, [&](int t) { return a.grad[t]; },
               [&](int t, float g) { a.grad[t] = static_cast<float>(g * c); });
  }
}

// ---------------------------------------------------------------------------
// Preference loss: sequences 0 .. P-1 are the chosen answers, P .. 2P-1 the
// rejected ones.
// ---------------------------------------------------------------------------
struct PreferenceArgs {
  SeqArgs q;       // S = 2 P
  const float *lp, *ref;  // ref may be null
  int32_t kind, normalise;
  double beta, margin, smoothing, grad_scale;
  struct Part {
    double x;      // sum of lp - ref
    int32_t n;     // tokens
  };
  Part* part;      // [S * parts]
  int32_t* pairs;  // pairs that count; read if have_pairs
  int32_t have_pairs;
  float* stats;    // [3]
  float* rewards;  // [S]
  float* grad;     // [T]
};
using Part = PreferenceArgs::Part;

__device__ __forceinline__ Sum4 preference_part(const PreferenceArgs& a, int s, int y, int lane,
                                                int team) {
  int t0, t1;
  part_range(a.q, s, y, t0, t1);
  Sum4 v;
  v.zero();
  struct Token {
    float lp, ref;
    bool on;
  };
  each_token(t0, t1, lane, team,
             [&](int t) {
               return Token{a.lp[t], a.ref != nullptr ? a.ref[t] : 0.0f, counts(a.q, t)};
             },
             [&](int, const Token& k) {
               // fp64: long sums whose difference between two answers is small
               if (k.on) {
                 v.x += static_cast<double>(k.lp) - static_cast<double>(k.ref);
                 v.n += 1;
               }
             });
  return v;
}

// One answer: S and its tokens.  LDS: `part` lies there, where a load needs no
// others in flight.
template <bool LDS>
__device__ __forceinline__ Part answer(const PreferenceArgs& a, const Part* part, int s) {
  Part r = {0.0, 0};
  part += static_cast<size_t>(s) * a.q.parts;
  constexpr int kLoads = LDS ? 1 : 16;
  int y0 = 0;
  if (!LDS && a.q.parts == 1) {
    r = part[0];
    y0 = 1;
  }
  for (; y0 < a.q.parts; y0 += kLoads) {
    Part p[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (y0 + u < a.q.parts) p[u] = part[y0 + u];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (y0 + u < a.q.parts) {
        r.x += p[u].x;
        r.n += p[u].n;
      }
  }
  if (a.normalise && r.n > 0) r.x /= r.n;
  return r;
}

// Loss of a pair that counts and its derivative by D = S_chosen - S_rejected.
__device__ __forceinline__ double pair_loss(const PreferenceArgs& a, double diff, double& dl) {
  if (a.kind == FS_PREFERENCE_IPO) {
    const double t = diff - 0.5 / a.beta;
    dl = 2.0 * t;
    return t * t;
  }
  const double x = a.beta * diff - a.margin;
  if (a.kind == FS_PREFERENCE_HINGE) {
    dl = x < 1.0 ? -a.beta : 0.0;
    return fmax(1.0 - x, 0.0);
  }
  // -(1 - eps) log sigmoid(x) - eps log sigmoid(-x)
  const double l = log1p(exp(-fabs(x)));
  dl = a.beta * (a.smoothing - 1.0 / (1.0 + exp(x)));
  return (1.0 - a.smoothing) * (fmax(-x, 0.0) + l) + a.smoothing * (fmax(x, 0.0) + l);
}

// Gradient of each token of sequence s that counts.
template <bool LDS>
__device__ __forceinline__ float answer_weight(const PreferenceArgs& a, const Part* part, int s,
                                               int pairs) {
  const int P = a.q.S / 2;
  const int p = s < P ? s : s - P;
  const Part hi = answer<LDS>(a, part, p), lo = answer<LDS>(a, part, P + p);
  if (hi.n == 0 || lo.n == 0) return 0.0f;
  double dl;
  pair_loss(a, hi.x - lo.x, dl);
  dl *= a.grad_scale / max(pairs, 1);
  if (a.normalise) dl /= s < P ? hi.n : lo.n;
  return static_cast<float>(s < P ? dl : -dl);
}

template <int THREADS, bool LDS = false>
__device__ __forceinline__ int count_pairs(const PreferenceArgs& a, const Part* part) {
  const int P = a.q.S / 2;
  int n = 0;
  for (int p = threadIdx.x; p < P; p += THREADS)
    n += answer<LDS>(a, part, p).n > 0 && answer<LDS>(a, part, P + p).n > 0;
  return block_count<THREADS>(n, 0).x;
}

// Statistics and rewards, by one block.
template <int THREADS, bool LDS = false>
__device__ __forceinline__ void preference_stats(const PreferenceArgs& a, const Part* part,
                                                 int pairs) {
  const int P = a.q.S / 2;
  Sum4 v;  // x: loss, y: margin of rewards, k: pairs whose chosen answer scores higher
  v.zero();
  for (int p = threadIdx.x; p < P; p += THREADS) {
    const Part hi = answer<LDS>(a, part, p), lo = answer<LDS>(a, part, P + p);
    a.rewards[p] = static_cast<float>(a.beta * hi.x);
    a.rewards[P + p] = static_cast<float>(a.beta * lo.x);
    if (hi.n > 0 && lo.n > 0) {
      double dl;
      v.x += pair_loss(a, hi.x - lo.x, dl);
      v.y += a.beta * (hi.x - lo.x);
      v.k += hi.x > lo.x;
    }
  }
  v = block_sum<THREADS>(v);
  if (threadIdx.x == 0) {
    const double d = max(pairs, 1);
    a.stats[0] = static_cast<float>(v.x / d);
    a.stats[1] = static_cast<float>(v.k / d);
    a.stats[2] = static_cast<float>(v.y / d);
  }
}

__device__ __forceinline__ void preference_grad_part(const PreferenceArgs& a, int s, int y, float w,
                                                     int lane, int team) {
  int t0, t1;
  part_range(a.q, s, y, t0, t1);
  each_token(t0, t1, lane, team, [&](int t) { return counts(a.q, t); },
             [&](int t, bool on) { a.grad[t] = on ? w : 0.0f; });
}

template <int TEAM>
__global__ __launch_bounds__(kThreads) void preference_sums_kernel(PreferenceArgs a) {
  const int64_t item = item_of_thread<TEAM>();
  const bool in = item < static_cast<int64_t>(a.q.S) * a.q.parts;
  Sum4 v;
  v.zero();
  if (in)
    v = preference_part(a, static_cast<int>(item / a.q.parts), static_cast<int>(item % a.q.parts),
                        threadIdx.x % TEAM, TEAM);
  if constexpr (TEAM > kWaveSize) v = block_sum<kThreads>(v);
  else v.wave_sum();
  if (in && threadIdx.x % TEAM == 0) a.part[item] = Part{v.x, v.n};
}

__global__ __launch_bounds__(kOneBlockThreads) void preference_pairs_kernel(PreferenceArgs a) {
  const int n = count_pairs<kOneBlockThreads>(a, a.part);
  if (threadIdx.x == 0) *a.pairs = n;
}

// Gradients; the grid's last block takes the statistics.
template <int TEAM>
__global__ __launch_bounds__(kThreads) void preference_grad_kernel(PreferenceArgs a) {
  outside(a.q, a.grad, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x,
          static_cast<int64_t>(gridDim.x) * kThreads);
  const int pairs = a.have_pairs ? *a.pairs : count_pairs<kThreads>(a, a.part);
  if (blockIdx.x == gridDim.x - 1) {
    preference_stats<kThreads>(a, a.part, pairs);
    return;
  }
  const int64_t item = item_of_thread<TEAM>();
  if (item >= static_cast<int64_t>(a.q.S) * a.q.parts) return;
  const int s = static_cast<int>(item / a.q.parts), y = static_cast<int>(item % a.q.parts);
  preference_grad_part(a, s, y, answer_weight<false>(a, a.part, s, pairs), threadIdx.x % TEAM, TEAM);
}

__global__ __launch_bounds__(kOneBlockThreads) void preference_one_block_kernel(PreferenceArgs a) {
  __shared__ Part part[kOneBlockItems];
  __shared__ float weight[kOneBlockSequences];
  outside(a.q, a.grad, threadIdx.x, kOneBlockThreads);
  constexpr int kWaves = kOneBlockThreads / kWaveSize;
  const int wave = threadIdx.x / kWaveSize, lane = threadIdx.x % kWaveSize;
  const int Y = a.q.parts, items = a.q.S * Y;
  for (int i = wave; i < items; i += kWaves) {
    Sum4 v = preference_part(a, i / Y, i % Y, lane, kWaveSize);
    v.wave_sum();
    if (lane == 0) part[i] = Part{v.x, v.n};
  }
  __syncthreads();
  const int pairs = count_pairs<kOneBlockThreads, true>(a, part);
  if (threadIdx.x < static_cast<unsigned>(a.q.S))
    weight[threadIdx.x] = answer_weight<true>(a, part, threadIdx.x, pairs);
  preference_stats<kOneBlockThreads, true>(a, part, pairs);
  __syncthreads();
  for (int i = wave; i < items; i += kWaves)
    preference_grad_part(a, i / Y, i % Y, weight[i / Y], lane, kWaveSize);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
bool one_block(int64_t S, int64_t T) {
  return S == 0 || (T <= kOneBlockTokens && S <= kOneBlockSequences);
}

// Parts per sequence: enough that a few long sequences still spread over the
// device (or over one block's waves), one where there are sequences enough.
int32_t loss_parts(int64_t S, int64_t T) {
  if (S <= 0 || S >= 512) return 1;
  if (one_block(S, T)) {
    const int64_t waves = (kOneBlockThreads / kWaveSize + S - 1) / S, by = (T / S + 63) / 64;
    return static_cast<int32_t>(waves < by ? waves : by < 1 ? 1 : by);
  }
  const int64_t by_grid = (512 + S - 1) / S;
  const int64_t fill = (T / S + 511) / 512;  // no parts below 512 tokens
  const int64_t p = by_grid < fill ? by_grid : fill;
  return static_cast<int32_t>(p < 1 ? 1 : p > kMaxParts ? kMaxParts : p);
}

struct LossLayout {
  size_t head, count, part, total;
  LossLayout(int64_t S, int64_t T) {
    if (one_block(S, T)) {
      head = count = part = total = 0;
      return;
    }
    const size_t items = static_cast<size_t>(S) * loss_parts(S, T);
    head = 0;  // totals
    count = 256;
    part = count + round_up(sizeof(int32_t) * items, 256);
    total = part + round_up(sizeof(Sum4) * items, 256);
  }
};

struct LossGrid {
  bool wide;
  int64_t items;
  unsigned blocks;
  explicit LossGrid(const SeqArgs& q) {
    items = static_cast<int64_t>(q.S) * q.parts;
    // (parts of a sequence have kBlockTeamTokens or so)
    wide = items < kBlockTeamItems && q.T / q.S >= kBlockTeamTokens;
    constexpr int per = kThreads / kWaveSize;
    blocks = static_cast<unsigned>(wide ? items : (items + per - 1) / per);
  }
};

hipError_t launch_policy(PolicyArgs& a, hipStream_t stream) {
  if (one_block(a.q.S, a.q.T)) {
    policy_one_block_kernel<<<1, kOneBlockThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  const LossGrid g(a.q);
  if (g.wide) policy_counts_kernel<kThreads><<<g.blocks, kThreads, 0, stream>>>(a);
  else policy_counts_kernel<kWaveSize><<<g.blocks, kThreads, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.have_totals = g.items > kInBlockItems;
  if (a.have_totals) {
    policy_totals_kernel<<<1, kOneBlockThreads, 0, stream>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (g.wide) policy_kernel<kThreads><<<g.blocks, kThreads, 0, stream>>>(a);
  else policy_kernel<kWaveSize><<<g.blocks, kThreads, 0, stream>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  policy_stats_kernel<<<1, kOneBlockThreads, 0, stream>>>(a, g.blocks);
  return hipGetLastError();
}

hipError_t launch_preference(PreferenceArgs& a, hipStream_t stream) {
  if (one_block(a.q.S, a.q.T)) {
    preference_one_block_kernel<<<1, kOneBlockThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  const LossGrid g(a.q);
  if (g.wide) preference_sums_kernel<kThreads><<<g.blocks, kThreads, 0, stream>>>(a);
  else preference_sums_kernel<kWaveSize><<<g.blocks, kThreads, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.have_pairs = g.items > kInBlockItems;
  if (a.have_pairs) {
    preference_pairs_kernel<<<1, kOneBlockThreads, 0, stream>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (g.wide) preference_grad_kernel<kThreads><<<g.blocks + 1, kThreads, 0, stream>>>(a);
  else preference_grad_kernel<kWaveSize><<<g.blocks + 1, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

constexpr int32_t kMaxSequences = 1 << 20;

fs_status check_sequences(const char* who, int32_t S, int32_t T, const int32_t* cu) {
  if (S < 0 || T < 0)
    return fail(FS_ERR_INVALID_ARG, "%s: sequence and token counts must be >= 0 (got %d, %d)", who,
                S, T);
  if (S > kMaxSequences)
    return fail(FS_ERR_UNSUPPORTED, "%s: %d sequences exceed the %d one call can take", who, S,
                kMaxSequences);
  if (!cu) return fail(FS_ERR_INVALID_ARG, "%s: null cu_seqlens", who);
  if (!aligned(cu, 4))
    return fail(FS_ERR_INVALID_ARG, "%s: cu_seqlens must be 4-byte aligned", who);
  return FS_OK;
}

fs_status check_workspace(const char* who, void* workspace, size_t have, size_t need) {
  if (need == 0) return FS_OK;
  if (!workspace) return fail(FS_ERR_INVALID_ARG, "%s: null workspace", who);
  if (!aligned(workspace, 256))
    return fail(FS_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  if (have < need)
    return fail(FS_ERR_WORKSPACE, "%s: workspace of %zu bytes is below the %zu required", who, have,
                need);
  return FS_OK;
}

}  // namespace
}  // namespace fs

extern "C" {

FS_API size_t fs_loss_workspace_bytes(int32_t n_sequences, int32_t n_tokens) {
  if (n_sequences < 0 || n_tokens < 0 || n_sequences > fs::kMaxSequences) return 0;
  return fs::LossLayout(n_sequences, n_tokens).total;
}

FS_API fs_status fs_policy_loss(const float* logprob, const float* old_logprob,
                                const float* ref_logprob, const float* advantages,
                                const uint8_t* mask, const int32_t* cu_seqlens,
                                int32_t n_sequences, int32_t n_tokens,
                                int32_t advantage_per_token, double clip_low, double clip_high,
                                double dual_clip, double kl_coef, fs_kl_kind kl_kind,
                                fs_loss_reduction reduction, double grad_scale,
                                int32_t zero_outside, float* out_stats, float* out_grad,
                                void* workspace, size_t workspace_bytes, void* stream) {
  using namespace fs;
  const char* who = "fs_policy_loss";
  fs_status st = check_sequences(who, n_sequences, n_tokens, cu_seqlens);
  if (st != FS_OK) return st;
  if (!out_stats || !aligned(out_stats, 4))
    return fail(FS_ERR_INVALID_ARG, "%s: out_stats must be a 4-byte aligned device pointer", who);
  if (n_tokens > 0) {
    if (!logprob || !old_logprob || !out_grad)
      return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (!aligned(logprob, 4) || !aligned(old_logprob, 4) || !aligned(out_grad, 4))
      return fail(FS_ERR_INVALID_ARG, "%s: token arrays must be 4-byte aligned", who);
    if (ref_logprob && !aligned(ref_logprob, 4))
      return fail(FS_ERR_INVALID_ARG, "%s: ref_logprob must be 4-byte aligned", who);
  }
  if (advantage_per_token ? n_tokens > 0 : n_sequences > 0)
    if (!advantages || !aligned(advantages, 4))
      return fail(FS_ERR_INVALID_ARG, "%s: advantages must be a 4-byte aligned device pointer", who);
  if (!(clip_low >= 0.0 && clip_low < 1.0))
    return fail(FS_ERR_INVALID_ARG, "%s: clip_low must be in [0, 1) (got %g)", who, clip_low);
  if (!(clip_high >= 0.0) || std::isinf(clip_high))
    return fail(FS_ERR_INVALID_ARG, "%s: clip_high must be finite and >= 0 (got %g)", who, clip_high);
  if (!(dual_clip == 0.0 || (dual_clip > 1.0 && !std::isinf(dual_clip))))
    return fail(FS_ERR_INVALID_ARG, "%s: dual_clip must be 0 (off) or finite and > 1 (got %g)", who,
                dual_clip);
  if (!std::isfinite(kl_coef) || !std::isfinite(grad_scale))
    return fail(FS_ERR_INVALID_ARG, "%s: kl_coef and grad_scale must be finite", who);
  if (kl_kind != FS_KL_K1 && kl_kind != FS_KL_K2 && kl_kind != FS_KL_K3)
    return fail(FS_ERR_INVALID_ARG, "%s: unknown kl_kind %d", who, static_cast<int>(kl_kind));
  if (reduction != FS_TOKEN_MEAN && reduction != FS_SEQUENCE_MEAN)
    return fail(FS_ERR_INVALID_ARG, "%s: unknown reduction %d", who, static_cast<int>(reduction));
  const LossLayout lay(n_sequences, n_tokens);
  st = check_workspace(who, workspace, workspace_bytes, lay.total);
  if (st != FS_OK) return st;
  if (start_launches()) return injected_failure(who);
  char* ws = static_cast<char*>(workspace);
  PolicyArgs a;
  a.q = {cu_seqlens, mask, n_sequences, n_tokens, loss_parts(n_sequences, n_tokens),
         zero_outside != 0};
  a.lp = logprob;
  a.old = old_logprob;
  a.ref = ref_logprob;
  a.adv = advantages;
  a.adv_per_token = advantage_per_token != 0;
  a.kl_kind = kl_kind;
  a.seq_mean = reduction == FS_SEQUENCE_MEAN;
  a.log_high = std::log1p(clip_high);
  a.log_low = std::log1p(-clip_low);
  a.log_cap = dual_clip != 0.0 ? std::log(dual_clip) : INFINITY;
  a.high = static_cast<float>(1.0 + clip_high);
  a.low = static_cast<float>(1.0 - clip_low);
  a.cap = static_cast<float>(dual_clip);
  a.kl_coef = kl_coef;
  a.grad_scale = grad_scale;
  a.totals = reinterpret_cast<int2*>(ws + lay.head);
  a.have_totals = 0;
  a.count = reinterpret_cast<int32_t*>(ws + lay.count);
  a.part = reinterpret_cast<Sum4*>(ws + lay.part);
  a.stats = out_stats;
  a.grad = out_grad;
  const hipError_t e = launch_policy(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FS_OK : hip_fail(e, "policy loss launch");
}

FS_API fs_status fs_preference_loss(const float* logprob, const float* ref_logprob,
                                    const uint8_t* mask, const int32_t* cu_seqlens,
                                    int32_t n_pairs, int32_t n_tokens, fs_preference_kind kind,
                                    double beta, double margin, double label_smoothing,
                                    int32_t length_normalised, double grad_scale,
                                    int32_t zero_outside, float* out_stats, float* out_rewards,
                                    float* out_grad, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  using namespace fs;
  const char* who = "fs_preference_loss";
  if (n_pairs < 0 || n_pairs > kMaxSequences / 2)
    return fail(n_pairs < 0 ? FS_ERR_INVALID_ARG : FS_ERR_UNSUPPORTED,
                "%s: n_pairs must be in [0, %d] (got %d)", who, kMaxSequences / 2, n_pairs);
  fs_status st = check_sequences(who, 2 * n_pairs, n_tokens, cu_seqlens);
  if (st != FS_OK) return st;
  if (!out_stats || !aligned(out_stats, 4))
    return fail(FS_ERR_INVALID_ARG, "%s: out_stats must be a 4-byte aligned device pointer", who);
  if (n_pairs > 0 && (!out_rewards || !aligned(out_rewards, 4)))
    return fail(FS_ERR_INVALID_ARG, "%s: out_rewards must be a 4-byte aligned device pointer", who);
  if (n_tokens > 0) {
    if (!logprob || !out_grad) return fail(FS_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (!aligned(logprob, 4) || !aligned(out_grad, 4) || (ref_logprob && !aligned(ref_logprob, 4)))
      return fail(FS_ERR_INVALID_ARG, "%s: token arrays must be 4-byte aligned", who);
  }
  if (kind != FS_PREFERENCE_SIGMOID && kind != FS_PREFERENCE_HINGE && kind != FS_PREFERENCE_IPO)
    return fail(FS_ERR_INVALID_ARG, "%s: unknown kind %d", who, static_cast<int>(kind));
  if (!(beta > 0.0) || std::isinf(beta))
    return fail(FS_ERR_INVALID_ARG, "%s: beta must be positive and finite (got %g)", who, beta);
  if (!std::isfinite(margin) || !std::isfinite(grad_scale))
    return fail(FS_ERR_INVALID_ARG, "%s: margin and grad_scale must be finite", who);
  if (kind == FS_PREFERENCE_IPO && margin != 0.0)
    return fail(FS_ERR_INVALID_ARG, "%s: margin does not apply to the IPO loss", who);
  if (!(label_smoothing >= 0.0 && label_smoothing <= 0.5) ||
      (kind != FS_PREFERENCE_SIGMOID && label_smoothing != 0.0))
    return fail(FS_ERR_INVALID_ARG,
                "%s: label_smoothing must be in [0, 0.5], and 0 but for the sigmoid loss (got %g)",
                who, label_smoothing);
  const LossLayout lay(2 * n_pairs, n_tokens);
  st = check_workspace(who, workspace, workspace_bytes, lay.total);
  if (st != FS_OK) return st;
  if (start_launches()) return injected_failure(who);
  char* ws = static_cast<char*>(workspace);
  PreferenceArgs a;
  a.q = {cu_seqlens, mask, 2 * n_pairs, n_tokens, loss_parts(2 * n_pairs, n_tokens),
         zero_outside != 0};
  a.lp = logprob;
  a.ref = ref_logprob;
  a.kind = kind;
  a.normalise = length_normalised != 0;
  a.beta = beta;
  a.margin = margin;
  a.smoothing = label_smoothing;
  a.grad_scale = grad_scale;
  a.pairs = reinterpret_cast<int32_t*>(ws + lay.head);
  a.have_pairs = 0;
  a.part = reinterpret_cast<Part*>(ws + lay.part);
  a.stats = out_stats;
  a.rewards = out_rewards;
  a.grad = out_grad;
  const hipError_t e = launch_preference(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FS_OK : hip_fail(e, "preference loss launch");
}

}  // extern "C"
