// fs_clip.hip -- the global norm of many gradient tensors, and clipping by it.
//
//   norm  = sqrt(sum_i sum_j x_ij^2),   y_ij = x_ij * min(1, max / (norm + 1e-6))
//
// Each block sums the squares of one chunk (fp64 throughout: no gradient's
// square overflows, and a sum of 10^9 terms loses nothing), the chunks' sums
// are added in order, and each block scales its chunk; where nothing is to be
// scaled in place the blocks return at once.  A few chunks' sums are added by
// every scaling block for itself, which saves a launch; more by one block
// between the two steps.  Bound by HBM: one read for the norm, one read and one
// write for the scaling, since the scale is known only after the last element.
// 1.85 GB of bf16 on an MI355X: 265 us for the norm (7.0 TB/s) and 600 us for
// the scaling (6.2 TB/s, reads and writes); a copy of 2 GiB by torch runs at
// 4.9 TB/s.
// Tensors go to the device as tables in kernel arguments (fs_clip_tables.hpp), so
// that nothing is copied or kept.
#include <cmath>

#include "fs_clip_tables.hpp"
#include "fs_device.hpp"
#include "fs_internal.hpp"

namespace fs {
namespace {

// More input than this: the norm's blocks take four chunks each.
constexpr int64_t kManyBytes = kChunkBytes * 1024;
// Inputs beyond the memory-side cache are not found there by the second step:
// both then read past the caches (non-temporal: 1.85 GB 861 against 930 us);
// smaller ones are (64 MB 31 against 34 us).  Results are stored past them in
// either case (256 MB 115 against 146 us, equal for less).
constexpr int64_t kCachedBytes = int64_t{256} << 20;
// Chunks' sums that every scaling block adds up for itself; more are added by a
// launch of their own (32 MB of fp32, 512 sums: 9.5 us in the blocks, 9.8 by a
// launch; 64 MB: 19.4 and 17.8).
constexpr int32_t kInBlockSums = 512;

struct ClipItem {
  const void* in;
  void* out;
  int64_t beg, end;  // elements
  int32_t dtype;
};

// The block's tensor and elements.  Thread k looks at entry k; the one whose
// blocks hold this one publishes the entry.
__device__ __forceinline__ ClipItem clip_item(const ClipTable& t) {
  __shared__ ClipItem item;
  const int k = threadIdx.x, b = blockIdx.x;
  if (k < t.n && t.first[k] <= b && b < t.first[k + 1]) {
    const int d = t.dtype[k];
    const int64_t elems = t.chunk / type_bytes(d);
    const int64_t beg = (b - t.first[k]) * elems, end = beg + elems;
    item = {t.in[k], t.out[k], beg, end < t.numel[k] ? end : t.numel[k], d};
  }
  __syncthreads();
  return item;
}

template <int DT>
struct Elem;
template <>
struct Elem<FS_FP32> {
  using T = float;
  __device__ __forceinline__ static float get(T x) { return x; }
  __device__ __forceinline__ static T put(float x) { return x; }
};
template <>
struct Elem<FS_BF16> {
  using T = __bf16;
  __device__ __forceinline__ static float get(T x) { return static_cast<float>(x); }
  __device__ __forceinline__ static T put(float x) { return static_cast<__bf16>(x); }
};
template <>
struct Elem<FS_FP16> {
  using T = _Float16;
  __device__ __forceinline__ static float get(T x) { return static_cast<float>(x); }
  __device__ __forceinline__ static T put(float x) { return static_cast<_Float16>(x); }
};

template <bool NTL, class V>
__device__ __forceinline__ V load_vec(const void* p) {
  const V* q = static_cast<const V*>(p);
  return NTL ? __builtin_nontemporal_load(q) : *q;
}

template <int DT, bool NTL>
__device__ __forceinline__ double sum_squares(const ClipItem& it) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int N = kVec / sizeof(T);
  const T* p = static_cast<const T*>(it.in);
  double s[kUnroll] = {};
  int64_t i = it.beg;
  if ((reinterpret_cast<uintptr_t>(p + it.beg) & (kVec - 1)) == 0) {
    typedef T V __attribute__((ext_vector_type(N)));
    constexpr int64_t kStep = static_cast<int64_t>(kClipThreads) * N;
    for (; i + kUnroll * kStep <= it.end; i += kUnroll * kStep) {
      V v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        v[u] = load_vec<NTL, V>(p + i + u * kStep + threadIdx.x * N);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const double x = E::get(v[u][j]);
          s[u] = __builtin_fma(x, x, s[u]);
        }
    }
  }
  for (i += threadIdx.x; i < it.end; i += kClipThreads) {
    const double x = E::get(p[i]);
    s[0] = __builtin_fma(x, x, s[0]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

template <int THREADS>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[THREADS / kWave];
#pragma unroll
  for (int m = kWave / 2; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  if ((threadIdx.x & (kWave - 1)) == 0) s[threadIdx.x / kWave] = v;
  __syncthreads();
  double r = s[0];
#pragma unroll
  for (int w = 1; w < THREADS / kWave; ++w) r += s[w];
  return r;
}

template <bool NTL>
__global__ __launch_bounds__(kClipThreads) void squares_kernel(ClipTable t, double* part) {
  const ClipItem it = clip_item(t);
  const double s = it.dtype == FS_FP32   ? sum_squares<FS_FP32, NTL>(it)
                   : it.dtype == FS_BF16 ? sum_squares<FS_BF16, NTL>(it)
                                         : sum_squares<FS_FP16, NTL>(it);
  const double all = block_sum<kClipThreads>(s);
  if (threadIdx.x == 0) part[t.base + static_cast<int>(blockIdx.x)] = all;
}

constexpr int kCloseThreads = 1024;

// The factor for all elements from the chunks' sums, on every thread.
template <int THREADS>
__device__ __forceinline__ float close_norm(const double* part, int32_t n, float max_norm,
                                            float* out_norm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += THREADS) s += part[i];
  const double norm = sqrt(block_sum<THREADS>(s));
  if (out_norm != nullptr && threadIdx.x == 0) *out_norm = static_cast<float>(norm);
  const double c = static_cast<double>(max_norm) / (norm + 1e-6);
  return isfinite(norm) && c < 1.0 ? static_cast<float>(c) : 1.0f;
}

__global__ __launch_bounds__(kCloseThreads) void norm_kernel(const double* part, int32_t n,
                                                             float max_norm, float* out_norm,
                                                             float* scale) {
  const float c = close_norm<kCloseThreads>(part, n, max_norm, out_norm);
  if (threadIdx.x == 0) *scale = c;
}

template <int DT, bool NTL>
__device__ __forceinline__ void scale_chunk(const ClipItem& it, float c) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int N = kVec / sizeof(T);
  const T* p = static_cast<const T*>(it.in);
  T* q = static_cast<T*>(it.out);
  int64_t i = it.beg;
  if (((reinterpret_cast<uintptr_t>(p + it.beg) | reinterpret_cast<uintptr_t>(q + it.beg)) &
       (kVec - 1)) == 0) {
    typedef T V __attribute__((ext_vector_type(N)));
    constexpr int64_t kStep = static_cast<int64_t>(kClipThreads) * N;
    for (; i + kUnroll * kStep <= it.end; i += kUnroll * kStep) {
      V v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        v[u] = load_vec<NTL, V>(p + i + u * kStep + threadIdx.x * N);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[u][j] = E::put(E::get(v[u][j]) * c);
        __builtin_nontemporal_store(v[u],
                                    reinterpret_cast<V*>(q + i + u * kStep + threadIdx.x * N));
      }
    }
  }
  for (i += threadIdx.x; i < it.end; i += kClipThreads) q[i] = E::put(E::get(p[i]) * c);
}

// part == null: the factor is in *scale; else from the n sums, and the first
// launch's first block writes the norm.
template <bool NTL>
__global__ __launch_bounds__(kClipThreads) void scale_kernel(ClipTable t, const float* scale,
                                                             const double* part, int32_t n,
                                                             float max_norm, float* out_norm) {
  const float c = part == nullptr ? *scale
                                  : close_norm<kClipThreads>(part, n, max_norm,
                                                             t.base + static_cast<int>(blockIdx.x) == 0
                                                                 ? out_norm : nullptr);
  const ClipItem it = clip_item(t);
  if (c == 1.0f && it.in == it.out) return;  // nothing to change (uniform)
  if (it.dtype == FS_FP32) scale_chunk<FS_FP32, NTL>(it, c);
  else if (it.dtype == FS_BF16) scale_chunk<FS_BF16, NTL>(it, c);
  else scale_chunk<FS_FP16, NTL>(it, c);
}

constexpr size_t kScaleBytes = 256;

size_t clip_workspace(int64_t chunks) {
  return kScaleBytes + round_up(sizeof(double) * static_cast<size_t>(chunks), 256);
}

}  // namespace
}  // namespace fs

extern "C" {

FS_API size_t fs_clip_grad_norm_workspace_bytes(const int64_t* numel, int32_t n) {
  const int64_t c = fs::max_chunks(numel, n);
  return c < 0 ? 0 : fs::clip_workspace(c);
}

FS_API fs_status fs_clip_grad_norm(const void* const* grads, void* const* out,
                                   const int64_t* numel, const fs_dtype* dtypes, int32_t n,
                                   float max_norm, float* out_norm, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  using namespace fs;
  const char* who = "fs_clip_grad_norm";
  if (n < 0 || n > kMaxTensors)
    return fail(FS_ERR_INVALID_ARG, "%s: n must be in [0, %d] (got %d)", who, kMaxTensors, n);
  if (n > 0 && (!grads || !numel || !dtypes))
    return fail(FS_ERR_INVALID_ARG, "%s: null host array", who);
  for (int32_t i = 0; i < n; ++i) {
    if (dtypes[i] != FS_BF16 && dtypes[i] != FS_FP16 && dtypes[i] != FS_FP32)
      return fail(FS_ERR_INVALID_ARG, "%s: unknown dtype %d of tensor %d", who,
                  static_cast<int>(dtypes[i]), i);
    if (numel[i] < 0)
      return fail(FS_ERR_INVALID_ARG, "%s: numel of tensor %d is negative", who, i);
    if (numel[i] == 0) continue;
    const size_t a = type_bytes(dtypes[i]);
    if (!grads[i] || !aligned(grads[i], a) || (out && (!out[i] || !aligned(out[i], a))))
      return fail(FS_ERR_INVALID_ARG, "%s: pointer of tensor %d is null or misaligned", who, i);
  }
  const int64_t chunks = max_chunks(numel, n);
  if (chunks < 0) return fail(FS_ERR_UNSUPPORTED, "%s: more elements than one call can take", who);
  if (!(max_norm >= 0.0f))
    return fail(FS_ERR_INVALID_ARG, "%s: max_norm must be >= 0 (got %g)", who, max_norm);
  if (!out_norm || !aligned(out_norm, 4))
    return fail(FS_ERR_INVALID_ARG, "%s: out_norm must be a 4-byte aligned device pointer", who);
  if (!workspace || !aligned(workspace, 256))
    return fail(FS_ERR_INVALID_ARG, "%s: workspace must be a 256-byte aligned device pointer", who);
  const size_t need = clip_workspace(chunks);
  if (workspace_bytes < need)
    return fail(FS_ERR_WORKSPACE, "%s: workspace of %zu bytes is below the %zu required", who,
                workspace_bytes, need);
  if (start_launches()) return injected_failure(who);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  float* scale = static_cast<float*>(workspace);
  double* part = reinterpret_cast<double*>(static_cast<char*>(workspace) + kScaleBytes);
  int64_t used = 0, bytes = 0;
  for (int32_t i = 0; i < n; ++i) bytes += numel[i] * type_bytes(dtypes[i]);
  const bool cached = bytes <= kCachedBytes;
  const int64_t norm_chunk = bytes <= kManyBytes ? kChunkBytes : 4 * kChunkBytes;
  hipError_t e = for_each_table(grads, out, numel, dtypes, n, norm_chunk,
                                [&](const ClipTable& t, unsigned b) {
    if (cached) squares_kernel<false><<<b, kClipThreads, 0, st>>>(t, part);
    else squares_kernel<true><<<b, kClipThreads, 0, st>>>(t, part);
    used += b;
    return hipGetLastError();
  });
  if (e != hipSuccess) return hip_fail(e, "gradient norm launch");
  const int32_t sums = static_cast<int32_t>(used);
  const bool norm_only = out == nullptr && std::isinf(max_norm);
  const bool in_blocks = sums > 0 && sums <= kInBlockSums && !norm_only;
  if (!in_blocks) {
    norm_kernel<<<1, kCloseThreads, 0, st>>>(part, sums, max_norm, out_norm, scale);
    if ((e = hipGetLastError()) != hipSuccess) return hip_fail(e, "gradient norm launch");
    if (norm_only) return FS_OK;
  }
  e = for_each_table(grads, out, numel, dtypes, n, kChunkBytes,
                     [&](const ClipTable& t, unsigned b) {
    const double* sums_or_null = in_blocks ? part : nullptr;
    if (cached)
      scale_kernel<false><<<b, kClipThreads, 0, st>>>(t, scale, sums_or_null, sums, max_norm, out_norm);
    else
      scale_kernel<true><<<b, kClipThreads, 0, st>>>(t, scale, sums_or_null, sums, max_norm, out_norm);
    return hipGetLastError();
  });
  return e == hipSuccess ? FS_OK : hip_fail(e, "gradient scaling launch");
}

}  // extern "C"
