// fs_fp8_quantize.hip -- bf16 weights and hidden states in 8-bit blocks.
#include "fs_fp8.hpp"
#include "fs_internal.hpp"

namespace fs {
namespace {

// Four waves per block of 128 x 128, four blocks side by side per thread block, so
// that a row is read 1 KB at a time, and neighbouring thread blocks along the rows.
// A wave has two groups of 16 rows; a lane holds, for each group and 64 columns, the
// 16 values that are its piece of the fragment order, in registers between the
// maximum and the conversion.  Bound by memory: two bytes read and one written per
// value.  128256 x 4096: 270 us, 5.8 TB/s (a copy runs at 5.2), stores past the caches;
// 283 by one wave per block, whose few waves also take 7 us on 1000 x 256 (5 here), 299
// with one block per thread block, 325 with neighbours down the columns.  Row-major,
// whose lanes store 64 bytes of a row at a time, 317.
constexpr int kQuantThreads = 1024;

template <bool PACKED>
__global__ __launch_bounds__(kQuantThreads) void quantize_weights_kernel(
    const __bf16* __restrict__ W, int32_t V, int32_t D, uint8_t* __restrict__ q,
    uint8_t* __restrict__ scale) {
  constexpr int kWaves = kQuantThreads / kWave, kAcross = kWaves / 4;
  constexpr int kGroups = 2, kSteps = kQuantBlock / 64;
  __shared__ uint32_t s_max[kWaves];
  const int lane = threadIdx.x & (kWave - 1), li = lane & 15, kb = lane >> 4;
  const int wave = threadIdx.x >> 6;
  const int KB = quant_blocks(D), across = (KB + kAcross - 1) / kAcross;
  const int cb = static_cast<int>(blockIdx.x % across) * kAcross + wave / 4;  // block of columns
  const int64_t vb = blockIdx.x / across;                                     // and of rows
  const int64_t group0 = vb * (kQuantBlock / 16) + wave % 4 * kGroups;
  const int k0 = cb * kQuantBlock + 16 * kb;
  u32x4 x[kGroups][kSteps][2];
  static_for<kGroups>([&](auto g) FS_INLINE {
    static_for<kSteps>([&](auto s) FS_INLINE {
      const int64_t v = (group0 + static_cast<int>(g)) * 16 + li;
      const int k = k0 + 64 * static_cast<int>(s);
      static_for<2>([&](auto j) FS_INLINE {
        const int kj = k + 8 * static_cast<int>(j);
        x[g][s][j] = u32x4{0u, 0u, 0u, 0u};
        if (v < V && kj < D) x[g][s][j] = *reinterpret_cast<const u32x4*>(W + v * D + kj);
      });
    });
  });
  auto fold = [&](auto f) FS_INLINE {
    static_for<kGroups>([&](auto g) FS_INLINE {
      static_for<kSteps>([&](auto s) FS_INLINE {
        static_for<2>([&](auto j) FS_INLINE {
          static_for<4>([&](auto c) FS_INLINE { f(x[g][s][j][decltype(c)::value]); });
        });
      });
    });
  };
  u16x2 any = {0, 0};
  fold([&](uint32_t pair) FS_INLINE { any = any_max2(any, pair); });
  uint32_t m = max(static_cast<uint32_t>(any[0]), static_cast<uint32_t>(any[1]));
  if (__ballot(m >= 0x7F80) != 0) {  // something is not finite: once more without it
    m = 0;
    fold([&](uint32_t pair) FS_INLINE { m = finite_max2(m, pair); });
  }
#pragma unroll
  for (int d = kWave / 2; d >= 1; d >>= 1)
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, kWave)));
  if (lane == 0) s_max[wave] = m;
  __syncthreads();
  if (cb >= KB) return;
  const int w0 = wave / 4 * 4;
  m = max(max(s_max[w0], s_max[w0 + 1]), max(s_max[w0 + 2], s_max[w0 + 3]));
  const int byte = scale_byte(m);
  const float down = scale_down(byte);
  if (lane == 0 && wave % 4 == 0) scale[vb * KB + cb] = static_cast<uint8_t>(byte);
  static_for<kGroups>([&](auto g) FS_INLINE {
    static_for<kSteps>([&](auto s) FS_INLINE {
      const u32x4 a = x[g][s][0], b = x[g][s][1];
      const u32x4 y = {to_e4m3(a[0], a[1], down), to_e4m3(a[2], a[3], down),
                       to_e4m3(b[0], b[1], down), to_e4m3(b[2], b[3], down)};
      const int64_t group = group0 + static_cast<int>(g);
      const int k = k0 + 64 * static_cast<int>(s);
      if constexpr (PACKED) {  // (D is a multiple of 64)
        const int step = cb * kSteps + static_cast<int>(s);
        if (group * 16 < V && step < D / 64)
          __builtin_nontemporal_store(
              y, reinterpret_cast<u32x4*>(q + (group * (D / 64) + step) * 1024 + lane * 16));
      } else {
        const int64_t v = group * 16 + li;
        if (v < V) {
          uint64_t* p = reinterpret_cast<uint64_t*>(q + v * D + k);
          if (D % 16 == 0) {
            if (k < D) __builtin_nontemporal_store(y, reinterpret_cast<u32x4*>(p));
          } else {
            if (k < D) p[0] = y[0] | static_cast<uint64_t>(y[1]) << 32;
            if (k + 8 < D) p[1] = y[2] | static_cast<uint64_t>(y[3]) << 32;
          }
        }
      }
    });
  });
}

// One thread per 16 bytes of the fragment order.  Bound by memory (128256 x 4096: 199 us,
// 5.3 TB/s read and written).
__global__ __launch_bounds__(256) void pack_fp8_kernel(const uint8_t* __restrict__ q, int32_t V,
                                                       int32_t D, int64_t pieces,
                                                       uint8_t* __restrict__ packed) {
  const int64_t steps = D / 64;
  for (int64_t p = blockIdx.x * 256ll + threadIdx.x; p < pieces; p += 256ll * gridDim.x) {
    const int lane = static_cast<int>(p & (kWave - 1));
    const int64_t gs = p >> 6, s = gs % steps, g = gs / steps;
    const int64_t v = g * 16 + (lane & 15);
    u32x4 x = {0u, 0u, 0u, 0u};
    if (v < V) x = *reinterpret_cast<const u32x4*>(q + v * D + 64 * s + 16 * (lane >> 4));
    *reinterpret_cast<u32x4*>(packed + p * 16) = x;
  }
}

// Hidden states: one block per row, a thread per 16 columns, eight per 128.
// TARGETS: also the logit of the row's token, with exact products summed in fp32.  The
// tiles' instructions round theirs (fs_fp8_tile.hpp), which the log-sum-exp over
// the other rows averages out but a single logit shows.  777 rows of 8192: 6 us; 1777
// rows of 5120 with targets 16, bound by memory: a row's pieces of 16 bytes lie 256
// apart in W, each in a line of its own.
template <bool TARGETS>
__global__ __launch_bounds__(1024) void quantize_rows_kernel(Fp8Args a) {
  static_assert(kMaxFp8D <= 1024 * 16, "a thread per 16 columns");
  __shared__ float s_sum[1024 / kWave];
  const int b = blockIdx.x, lane = threadIdx.x & (kWave - 1), k = 16 * static_cast<int>(threadIdx.x);
  const bool in = k < a.D;  // (D is a multiple of 64: sixteen columns are all inside or all past it)
  u32x4 x[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
  if (in) {
    const u32x4* p = reinterpret_cast<const u32x4*>(a.h + static_cast<int64_t>(b) * a.D + k);
    x[0] = p[0];
    x[1] = p[1];
  }
  int loc = -1, wbyte = 127;
  u32x4 w = {0u, 0u, 0u, 0u};
  if constexpr (TARGETS) {
    loc = target_row(a.ids[b], a.vocab_offset, a.V);
    if (loc >= 0 && in) {
      const size_t step = static_cast<size_t>(loc / 16) * (a.D / 64) + k / 64;
      w = *reinterpret_cast<const u32x4*>(a.w + (step * 64 + loc % 16 + 16 * (k / 16 % 4)) * 16);
      wbyte = a.wscale[static_cast<size_t>(loc / kQuantBlock) * a.KB + k / kQuantBlock];
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) m = finite_max2(m, x[j][c]);
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1)
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, kWave)));
  const int byte = scale_byte(m);
  const float down = scale_down(byte);
  const u32x4 y = {to_e4m3(x[0][0], x[0][1], down), to_e4m3(x[0][2], x[0][3], down),
                   to_e4m3(x[1][0], x[1][1], down), to_e4m3(x[1][2], x[1][3], down)};
  if (k < a.Dp) {
    *reinterpret_cast<u32x4*>(a.hq + static_cast<int64_t>(b) * a.Dp + k) = y;
    if (threadIdx.x % 8 == 0)
      a.hscale[static_cast<int64_t>(k / kQuantBlock) * a.Bp + b] = static_cast<uint8_t>(byte);
  }
  if constexpr (TARGETS) {
    if (loc < 0) return;  // (block-uniform)
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bf16x8 p = widen(y[2 * j], y[2 * j + 1], scale_up(byte));
      const bf16x8 q = widen(w[2 * j], w[2 * j + 1], scale_up(wbyte));
#pragma unroll
      for (int c = 0; c < 8; ++c)
        z = __builtin_fmaf(static_cast<float>(p[c]), static_cast<float>(q[c]), z);
    }
#pragma unroll
    for (int d = kWave / 2; d >= 1; d >>= 1) z += __shfl_xor(z, d, kWave);
    if (lane == 0) s_sum[threadIdx.x / kWave] = z;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int v = 1; v < static_cast<int>(blockDim.x) / kWave; ++v) z += s_sum[v];
      a.target[b] = z * score_inv_t(a.temperature, b);
    }
  }
}

}  // namespace

hipError_t launch_quantize_weights(const __bf16* W, int32_t V, int32_t D, bool packed, uint8_t* q,
                                   uint8_t* scale, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(quant_blocks(V)) * ((quant_blocks(D) + 3) / 4);
  if (packed) quantize_weights_kernel<true><<<grid, kQuantThreads, 0, stream>>>(W, V, D, q, scale);
  else quantize_weights_kernel<false><<<grid, kQuantThreads, 0, stream>>>(W, V, D, q, scale);
  return hipGetLastError();
}

hipError_t launch_pack_fp8(const uint8_t* q, int32_t V, int32_t D, uint8_t* packed,
                           hipStream_t stream) {
  const int64_t pieces = static_cast<int64_t>(fp8_groups(V)) * (D / 64) * kWave;
  const int64_t blocks = (pieces + 255) / 256;
  pack_fp8_kernel<<<static_cast<unsigned>(blocks < 65536 ? blocks : 65536), 256, 0, stream>>>(
      q, V, D, pieces, packed);
  return hipGetLastError();
}

hipError_t launch_quantize_rows(const Fp8Args& a, hipStream_t stream) {
  const unsigned threads = static_cast<unsigned>(round_up(a.Dp / 16, kWave));
  if (a.ids != nullptr) quantize_rows_kernel<true><<<a.B, threads, 0, stream>>>(a);
  else quantize_rows_kernel<false><<<a.B, threads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace fs
