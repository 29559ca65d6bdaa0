// fs_loss.hip -- losses on token log-probabilities, with their gradients: the
// clipped policy loss with a KL penalty, and the preference loss of paired
// answers.
//
// Both read a packed batch of sequences (tokens [cu[s], cu[s+1]) of flat
// arrays) and run in three phases, because every token's gradient carries a
// count over the whole batch (tokens, sequences or pairs that count):
//   sums    one team of threads per part of a sequence: fp64 sums over its
//           unmasked tokens into the workspace
//   close   one block: each sequence's weight, the loss and the statistics
//   grad    the teams again: each token's gradient from its sequence's weight
// Every sum is taken in a fixed order (strided lanes, shuffles, then parts in
// order): no atomics, so equal calls give equal bits.  A token is 13 to 21
// bytes and a few dozen operations, so a batch of any usual size is bound by
// launches and memory latency, not by bandwidth.
#include <cmath>

#include "fs_host.hpp"
#include "fs_internal.hpp"

namespace fs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaveSize = 64;
constexpr int kOneBlockThreads = 1024;

struct SeqArgs {
  const int32_t* cu;     // [S + 1]
  const uint8_t* mask;   // [T] or null
  int32_t S, T;
  int32_t parts;         // parts per sequence
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
  for (int w = 1; w < THREADS / kWaveSize; ++w) r.add(s[w]);
  __syncthreads();
  return r;
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
  Sum4* part;      // [S][parts]
  float* weight;   // [S]
  float* stats;    // [4]
  float* grad;     // [T]
};

struct TokenTerms {
  float surr, kl, gs, gk;
  bool clipped;
};

__device__ __forceinline__ TokenTerms policy_token(const PolicyArgs& a, int t, float A) {
  TokenTerms o;
  const double lp = a.lp[t];
  const double d = lp - static_cast<double>(a.old[t]);
  const float r = expf(static_cast<float>(d));
  const bool over = d > a.log_high, under = d < a.log_low;
  const bool cap = A < 0.0f && d > a.log_cap;
  o.clipped = (A > 0.0f && over) || (A < 0.0f && under) || cap;
  const float rc = cap ? a.cap : over ? a.high : under ? a.low : r;
  // an advantage of zero leaves nothing, whatever the ratio
  const float live = A == 0.0f ? 0.0f : -(r * A);
  o.surr = o.clipped ? -(rc * A) : live;
  o.gs = o.clipped ? 0.0f : live;
  o.kl = o.gk = 0.0f;
  if (a.ref != nullptr) {
    const double e = static_cast<double>(a.ref[t]) - lp;
    if (a.kl_kind == FS_KL_K1) {
      o.kl = static_cast<float>(-e);
      o.gk = 1.0f;
    } else if (a.kl_kind == FS_KL_K2) {
      o.kl = static_cast<float>(0.5 * e * e);
      o.gk = static_cast<float>(-e);
    } else {
      // e^q - q - 1 cancels to q^2 / 2 near 0: in fp64
      const double x = expm1(e);
      o.kl = static_cast<float>(x - e);
      o.gk = static_cast<float>(-x);
    }
  }
  return o;
}

// Sums of part y of sequence s over a team of `team` threads, lane in [0, team).
__device__ __forceinline__ Sum4 policy_part(const PolicyArgs& a, int s, int y, int lane, int team) {
  int t0, t1;
  part_range(a.q, s, y, t0, t1);
  Sum4 v;
  v.zero();
  const float As = a.adv_per_token ? 0.0f : a.adv[s];
  for (int t = t0 + lane; t < t1; t += team) {
    if (!counts(a.q, t)) continue;  // masked tokens may hold anything
    const TokenTerms o = policy_token(a, t, a.adv_per_token ? a.adv[t] : As);
    v.x += static_cast<double>(o.surr);
    v.y += static_cast<double>(o.kl);
    v.n += 1;
    v.k += o.clipped ? 1 : 0;
  }
  return v;
}

__device__ __forceinline__ void policy_grad_part(const PolicyArgs& a, int s, int y, int lane,
                                                 int team) {
  int t0, t1;
  part_range(a.q, s, y, t0, t1);
  const float w = a.weight[s], k = static_cast<float>(a.kl_coef);
  const float As = a.adv_per_token ? 0.0f : a.adv[s];
  for (int t = t0 + lane; t < t1; t += team) {
    float g = 0.0f;
    if (counts(a.q, t)) {
      const TokenTerms o = policy_token(a, t, a.adv_per_token ? a.adv[t] : As);
      g = (o.gs + k * o.gk) * w;
    }
    a.grad[t] = g;
  }
}

// Weights and statistics, by one block of THREADS threads.
template <int THREADS>
__device__ __forceinline__ void policy_close(const PolicyArgs& a) {
  const int S = a.q.S, Y = a.q.parts;
  Sum4 v;
  v.zero();
  int filled = 0;
  for (int s = threadIdx.x; s < S; s += THREADS) {
    Sum4 one;
    one.zero();
    for (int y = 0; y < Y; ++y) one.add(a.part[static_cast<size_t>(s) * Y + y]);
    if (one.n > 0) ++filled;
    if (a.seq_mean && one.n > 0) {
      one.x /= one.n;
      one.y /= one.n;
    }
    v.add(one);
  }
  const Sum4 all = block_sum<THREADS>(v);
  Sum4 f;
  f.zero();
  f.n = filled;
  const int groups = block_sum<THREADS>(f).n;
  const double denom = a.seq_mean ? max(groups, 1) : max(all.n, 1);
  for (int s = threadIdx.x; s < S; s += THREADS) {
    double w = 1.0 / denom;
    if (a.seq_mean) {
      int n = 0;
      for (int y = 0; y < Y; ++y) n += a.part[static_cast<size_t>(s) * Y + y].n;
      w /= max(n, 1);
    }
    a.weight[s] = static_cast<float>(w * a.grad_scale);
  }
  if (threadIdx.x == 0) {
    const double surr = all.x / denom, kl = all.y / denom;
    a.stats[0] = static_cast<float>(surr + a.kl_coef * kl);
    a.stats[1] = static_cast<float>(surr);
    a.stats[2] = static_cast<float>(kl);
    a.stats[3] = static_cast<float>(static_cast<double>(all.k) / max(all.n, 1));
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
  double beta, margin, smoothing;
  double grad_scale;
  Sum4* part;      // [2P][parts]: x the sum of lp - ref, n the tokens
  float* weight;   // [2P]: each token's gradient
  float* stats;    // [3]
  float* rewards;  // [2P]
  float* grad;     // [T]
};

__device__ __forceinline__ Sum4 preference_part(const PreferenceArgs& a, int s, int y, int lane,
                                                int team) {
  int t0, t1;
  part_range(a.q, s, y, t0, t1);
  Sum4 v;
  v.zero();
  for (int t = t0 + lane; t < t1; t += team) {
    if (!counts(a.q, t)) continue;
    // fp64: long sums whose difference between two answers is small
    v.x += static_cast<double>(a.lp[t]) - (a.ref ? static_cast<double>(a.ref[t]) : 0.0);
    v.n += 1;
  }
  return v;
}

__device__ __forceinline__ void preference_grad_part(const PreferenceArgs& a, int s, int y,
                                                     int lane, int team) {
  int t0, t1;
  part_range(a.q, s, y, t0, t1);
  const float w = a.weight[s];
  for (int t = t0 + lane; t < t1; t += team) a.grad[t] = counts(a.q, t) ? w : 0.0f;
}

template <int THREADS>
__device__ __forceinline__ void preference_close(const PreferenceArgs& a) {
  const int P = a.q.S / 2, Y = a.q.parts;
  auto gather = [&](int s) {
    Sum4 one;
    one.zero();
    for (int y = 0; y < Y; ++y) one.add(a.part[static_cast<size_t>(s) * Y + y]);
    if (a.normalise && one.n > 0) one.x /= one.n;
    return one;
  };
  Sum4 c;
  c.zero();
  for (int p = threadIdx.x; p < P; p += THREADS)
    if (gather(p).n > 0 && gather(P + p).n > 0) ++c.n;
  const double pairs = max(block_sum<THREADS>(c).n, 1);
  Sum4 v;  // x: loss, y: margin of rewards, k: pairs whose chosen answer scores higher
  v.zero();
  for (int p = threadIdx.x; p < P; p += THREADS) {
    const Sum4 hi = gather(p), lo = gather(P + p);
    a.rewards[p] = static_cast<float>(a.beta * hi.x);
    a.rewards[P + p] = static_cast<float>(a.beta * lo.x);
    double dl = 0.0;
    if (hi.n > 0 && lo.n > 0) {
      const double diff = hi.x - lo.x;
      if (a.kind == FS_PREFERENCE_IPO) {
        const double t = diff - 0.5 / a.beta;
        v.x += t * t;
        dl = 2.0 * t;
      } else {
        const double x = a.beta * diff - a.margin;
        if (a.kind == FS_PREFERENCE_HINGE) {
          v.x += fmax(1.0 - x, 0.0);
          dl = x < 1.0 ? -a.beta : 0.0;
        } else {
          // -(1 - eps) log sigmoid(x) - eps log sigmoid(-x)
          const double l = log1p(exp(-fabs(x)));
          v.x += (1.0 - a.smoothing) * (fmax(-x, 0.0) + l) + a.smoothing * (fmax(x, 0.0) + l);
          dl = a.beta * (a.smoothing - 1.0 / (1.0 + exp(x)));
        }
      }
      v.y += a.beta * diff;
      v.k += diff > 0.0 ? 1 : 0;
      dl *= a.grad_scale / pairs;
    }
    const int nh = a.normalise ? max(hi.n, 1) : 1, nl = a.normalise ? max(lo.n, 1) : 1;
    a.weight[p] = static_cast<float>(dl / nh);
    a.weight[P + p] = static_cast<float>(-dl / nl);
  }
  const Sum4 all = block_sum<THREADS>(v);
  if (threadIdx.x == 0) {
    a.stats[0] = static_cast<float>(all.x / pairs);
    a.stats[1] = static_cast<float>(all.k / pairs);
    a.stats[2] = static_cast<float>(all.y / pairs);
  }
}

// ---------------------------------------------------------------------------
// The two losses behind one set of kernels.
// ---------------------------------------------------------------------------
struct Policy {
  using Args = PolicyArgs;
  __device__ __forceinline__ static Sum4 part(const Args& a, int s, int y, int lane, int team) {
    return policy_part(a, s, y, lane, team);
  }
  __device__ __forceinline__ static void grad(const Args& a, int s, int y, int lane, int team) {
    policy_grad_part(a, s, y, lane, team);
  }
  template <int THREADS>
  __device__ __forceinline__ static void close(const Args& a) { policy_close<THREADS>(a); }
};

struct Preference {
  using Args = PreferenceArgs;
  __device__ __forceinline__ static Sum4 part(const Args& a, int s, int y, int lane, int team) {
    return preference_part(a, s, y, lane, team);
  }
  __device__ __forceinline__ static void grad(const Args& a, int s, int y, int lane, int team) {
    preference_grad_part(a, s, y, lane, team);
  }
  template <int THREADS>
  __device__ __forceinline__ static void close(const Args& a) { preference_close<THREADS>(a); }
};

// TEAM threads per part: a wave each for short sequences, a block for long ones.
template <class L, int TEAM>
__global__ __launch_bounds__(kThreads) void loss_sums_kernel(typename L::Args a) {
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / TEAM) + threadIdx.x / TEAM;
  const int64_t items = static_cast<int64_t>(a.q.S) * a.q.parts;
  if constexpr (TEAM == kThreads) {
    const int s = static_cast<int>(item / a.q.parts), y = static_cast<int>(item % a.q.parts);
    const Sum4 v = block_sum<kThreads>(L::part(a, s, y, threadIdx.x, TEAM));
    if (threadIdx.x == 0) a.part[item] = v;
  } else {
    if (item >= items) return;  // uniform per wave
    const int s = static_cast<int>(item / a.q.parts), y = static_cast<int>(item % a.q.parts);
    Sum4 v = L::part(a, s, y, threadIdx.x % TEAM, TEAM);
    v.wave_sum();
    if (threadIdx.x % TEAM == 0) a.part[item] = v;
  }
}

template <class L>
__global__ __launch_bounds__(kOneBlockThreads) void loss_close_kernel(typename L::Args a) {
  L::template close<kOneBlockThreads>(a);
}

template <class L, int TEAM>
__global__ __launch_bounds__(kThreads) void loss_grad_kernel(typename L::Args a) {
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / TEAM) + threadIdx.x / TEAM;
  if (item >= static_cast<int64_t>(a.q.S) * a.q.parts) return;
  L::grad(a, static_cast<int>(item / a.q.parts), static_cast<int>(item % a.q.parts),
          threadIdx.x % TEAM, TEAM);
}

// The three phases in one block, for batches that one block reads in about
// the time of the two further launches.
template <class L>
__global__ __launch_bounds__(kOneBlockThreads) void loss_one_block_kernel(typename L::Args a) {
  const int wave = threadIdx.x / kWaveSize, lane = threadIdx.x % kWaveSize;
  constexpr int kWaves = kOneBlockThreads / kWaveSize;
  const int items = a.q.S * a.q.parts;
  for (int i = wave; i < items; i += kWaves) {
    Sum4 v = L::part(a, i / a.q.parts, i % a.q.parts, lane, kWaveSize);
    v.wave_sum();
    if (lane == 0) a.part[i] = v;
  }
  __syncthreads();
  L::template close<kOneBlockThreads>(a);
  __syncthreads();
  for (int i = wave; i < items; i += kWaves)
    L::grad(a, i / a.q.parts, i % a.q.parts, lane, kWaveSize);
}

// Tokens one block handles by itself, and the sequences' mean length from
// which a part takes a block rather than a wave.
constexpr int64_t kOneBlockTokens = 4096;
constexpr int64_t kBlockTeamTokens = 512;
// Tokens per part of long sequences, and the most parts of one.
constexpr int64_t kPartTokens = 4096;
constexpr int32_t kMaxParts = 256;

// Parts per sequence: enough that a few long sequences still spread over the
// device, one where there are sequences enough.
int32_t loss_parts(int64_t S, int64_t T) {
  if (S <= 0 || S >= 512) return 1;
  if (T <= kOneBlockTokens) {  // one block: a part for each of its waves
    const int64_t waves = (kOneBlockThreads / kWaveSize + S - 1) / S, by = (T / S + 63) / 64;
    return static_cast<int32_t>(waves < by ? waves : by < 1 ? 1 : by);
  }
  const int64_t by_len = (T / S + kPartTokens - 1) / kPartTokens;
  const int64_t by_grid = (512 + S - 1) / S;
  const int64_t fill = (T / S + 511) / 512;  // no parts below 512 tokens
  int64_t p = by_len > by_grid ? by_len : by_grid;
  p = p < fill ? p : fill;
  return static_cast<int32_t>(p < 1 ? 1 : p > kMaxParts ? kMaxParts : p);
}

size_t part_bytes(int64_t S, int64_t T) {
  return round_up(sizeof(Sum4) * static_cast<size_t>(S) * loss_parts(S, T), 256);
}

size_t loss_workspace(int64_t S, int64_t T) {
  return part_bytes(S, T) + round_up(sizeof(float) * static_cast<size_t>(S), 256);
}

template <class L>
hipError_t launch_loss(const typename L::Args& a, hipStream_t stream) {
  const int64_t S = a.q.S, T = a.q.T, items = S * a.q.parts;
  if (S == 0 || (T <= kOneBlockTokens && S <= kOneBlockTokens)) {
    loss_one_block_kernel<L><<<1, kOneBlockThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  const bool wide = T / S >= kBlockTeamTokens;
  constexpr int per = kThreads / kWaveSize;
  const dim3 grid(static_cast<unsigned>(wide ? items : (items + per - 1) / per));
  if (wide) loss_sums_kernel<L, kThreads><<<grid, kThreads, 0, stream>>>(a);
  else loss_sums_kernel<L, kWaveSize><<<grid, kThreads, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  loss_close_kernel<L><<<1, kOneBlockThreads, 0, stream>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (wide) loss_grad_kernel<L, kThreads><<<grid, kThreads, 0, stream>>>(a);
  else loss_grad_kernel<L, kWaveSize><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

constexpr int32_t kMaxSequences = 1 << 24;

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
  const size_t b = fs::loss_workspace(n_sequences, n_tokens);
  return b < 256 ? 256 : b;
}

FS_API fs_status fs_policy_loss(const float* logprob, const float* old_logprob,
                                const float* ref_logprob, const float* advantages,
                                const uint8_t* mask, const int32_t* cu_seqlens,
                                int32_t n_sequences, int32_t n_tokens,
                                int32_t advantage_per_token, double clip_low, double clip_high,
                                double dual_clip, double kl_coef, fs_kl_kind kl_kind,
                                fs_loss_reduction reduction, double grad_scale, float* out_stats,
                                float* out_grad, void* workspace, size_t workspace_bytes,
                                void* stream) {
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
  st = check_workspace(who, workspace, workspace_bytes, loss_workspace(n_sequences, n_tokens));
  if (st != FS_OK) return st;
  if (start_launches()) return injected_failure(who);
  PolicyArgs a;
  a.q = {cu_seqlens, mask, n_sequences, n_tokens, loss_parts(n_sequences, n_tokens)};
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
  a.part = static_cast<Sum4*>(workspace);
  a.weight = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      part_bytes(n_sequences, n_tokens));
  a.stats = out_stats;
  a.grad = out_grad;
  const hipError_t e = launch_loss<Policy>(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FS_OK : hip_fail(e, "policy loss launch");
}

FS_API fs_status fs_preference_loss(const float* logprob, const float* ref_logprob,
                                    const uint8_t* mask, const int32_t* cu_seqlens,
                                    int32_t n_pairs, int32_t n_tokens, fs_preference_kind kind,
                                    double beta, double margin, double label_smoothing,
                                    int32_t length_normalised, double grad_scale, float* out_stats,
                                    float* out_rewards, float* out_grad, void* workspace,
                                    size_t workspace_bytes, void* stream) {
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
  st = check_workspace(who, workspace, workspace_bytes, loss_workspace(2 * n_pairs, n_tokens));
  if (st != FS_OK) return st;
  if (start_launches()) return injected_failure(who);
  PreferenceArgs a;
  a.q = {cu_seqlens, mask, 2 * n_pairs, n_tokens, loss_parts(2 * n_pairs, n_tokens)};
  a.lp = logprob;
  a.ref = ref_logprob;
  a.kind = kind;
  a.normalise = length_normalised != 0;
  a.beta = beta;
  a.margin = margin;
  a.smoothing = label_smoothing;
  a.grad_scale = grad_scale;
  a.part = static_cast<Sum4*>(workspace);
  a.weight = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      part_bytes(2 * n_pairs, n_tokens));
  a.stats = out_stats;
  a.rewards = out_rewards;
  a.grad = out_grad;
  const hipError_t e = launch_loss<Preference>(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FS_OK : hip_fail(e, "preference loss launch");
}

}  // extern "C"
