// fs_fp8_stream.hpp -- the 8-bit LM head for up to 32 rows: logits, token scores
// or samples from one pass over W.  Instantiated in fs_fp8_stream_*.hip, which
// compile in parallel.
#pragma once

#include "fs_fp8.hpp"
#include "fs_sampler.hpp"

namespace fs {

// Bound by reading W once.  A block's NW waves split D (KS steps of 64 columns
// each, KS even: a wave holds whole blocks of 128) and keep their slice of h in
// registers; blocks sweep the 16-row vocabulary groups strided by the grid, so
// that the rows being read form a narrow moving window of W (HBM page locality),
// through a ring of P loads of 1 KB that runs ahead across groups.
//
// The products are bf16 ones: an e4m3 value times its power of two has four
// significant bits, so it is exact in bf16, and v_cvt_scalef32_pk_bf16_fp8 makes
// two of them in one instruction (7 us of the vector units' time for 128256 x
// 4096); what bounds the kernel is memory either way, and bf16 MFMAs add in fp32
// what 8-bit ones would round (fs_fp8_tile.hpp).  h is quantised as it is loaded:
// the four lanes that share a row hold a block's 128 columns between them.
//
// The partial sums of the waves meet in LDS, U groups at a time; the wave whose turn it
// is adds a group's in wave order and hands the 16 rows' logits to its output.  A block
// takes C neighbouring groups (a multiple of U), then those of the next sweep.
template <int OUT, int NT, int NW, int KS, int P, bool WHOLE, int C, int U>
__global__ __launch_bounds__(NW * kWave) void fp8_stream_kernel(Fp8Args a) {
  static_assert(KS % P == 0, "the load ring must tile a group");
  static_assert(KS % 2 == 0, "a wave holds whole blocks");
  static_assert(C % U == 0, "groups that meet are neighbours");
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn_smem[];
  f32x4* red = reinterpret_cast<f32x4*>(dyn_smem);  // [2][NW][U * NT][kWave]
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int li = lane & 15, kb = lane >> 4;
  const int G = gridDim.x, ngroups = (a.V - 1) / 16 + 1;
  const int steps = a.D / 64, step0 = wave * KS;

  // ---- h: quantised, then exact in bf16 ----
  bf16x8 hreg[KS][2][NT];
  float inv_t[NT];
  bool greedy[NT];
  int loc[NT];
  static_for<NT>([&](auto n) FS_INLINE {
    const int b = n * 16 + li, bc = min(b, a.B - 1);
    const __bf16* hp = a.h + static_cast<size_t>(bc) * a.D + 16 * kb;
    static_for<KS / 2>([&](auto i) FS_INLINE {
      u32x4 x[2][2];
      uint32_t m = 0;
      static_for<2>([&](auto s) FS_INLINE {
        const int step = step0 + 2 * static_cast<int>(i) + static_cast<int>(s);
        static_for<2>([&](auto j) FS_INLINE {
          x[s][j] = *reinterpret_cast<const u32x4*>(hp + 64 * min(step, steps - 1) + 8 * j);
          if (!WHOLE && step >= steps) x[s][j] = u32x4{0u, 0u, 0u, 0u};
          static_for<4>([&](auto c) FS_INLINE { m = finite_max2(m, x[s][j][decltype(c)::value]); });
        });
      });
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16, kWave)));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32, kWave)));
      const int byte = scale_byte(m);
      const float down = scale_down(byte), up = scale_up(byte);
      static_for<2>([&](auto s) FS_INLINE {
        static_for<2>([&](auto j) FS_INLINE {
          const u32x4 y = x[s][j];
          hreg[2 * decltype(i)::value + decltype(s)::value][j][n] =
              widen(to_e4m3(y[0], y[1], down), to_e4m3(y[2], y[3], down), up);
        });
      });
    });
    loc[n] = -1;
    inv_t[n] = 1.0f;
    greedy[n] = false;
    if constexpr (OUT == kTokenScores) {
      inv_t[n] = score_inv_t(a.temperature, bc);
      loc[n] = b < a.B ? target_row(a.ids[bc], a.vocab_offset, a.V) : -1;
    }
    if constexpr (OUT == kSamples) {
      const float T = a.temperature[bc];
      greedy[n] = row_is_greedy(T);
      inv_t[n] = row_inv_temperature(T);
    }
  });

  // The block's t-th group: C neighbouring ones, then those of the next sweep.
  auto nth = [&](int t) FS_INLINE {
    return (t / C * G + static_cast<int>(blockIdx.x)) * C + t % C;
  };
  // The lane's 16 bytes of the wave's step s of group t (clamped to the last group).
  auto group = [&](int t) FS_INLINE {
    return a.w + (static_cast<size_t>(min(t, ngroups - 1)) * steps + (WHOLE ? step0 : 0)) * 1024 +
           lane * 16;
  };
  auto load = [&](const uint8_t* p, int s) FS_INLINE {
    return __builtin_nontemporal_load(
        reinterpret_cast<const u32x4*>(p + (WHOLE ? s : min(step0 + s, steps - 1)) * 1024));
  };
  // The scales of the wave's blocks in group t's rows, one per lane.
  auto scales = [&](int t) FS_INLINE {
    const int block = min(step0 / 2 + min(lane, KS / 2 - 1), a.KB - 1);
    return static_cast<int>(a.wscale[static_cast<size_t>(min(t, ngroups - 1) / 8) * a.KB + block]);
  };
  const int whole_steps = __builtin_amdgcn_readfirstlane(min(max(steps - step0, 0), KS));

  const Philox philox(a.seed);
  ArgMax best[NT];
  float m[NT], s_[NT];
  static_for<NT>([&](auto n) FS_INLINE {
    best[n].init();
    m[n] = LseAcc::kMasked;
    s_[n] = 0.0f;
  });
  const uint8_t* wp = group(nth(0));
  const uint8_t* wn = group(nth(1));
  int sc = scales(nth(0)), sc_next = scales(nth(1));
  u32x4 ring[P];
  static_for<P>([&](auto p) FS_INLINE { ring[p] = load(wp, p); });
  for (int it = 0; nth(it * U) < ngroups; ++it) {
    f32x4 acc[U][NT];
    int live = whole_steps;
    if constexpr (!WHOLE) asm volatile("" : "+s"(live));  // (compared anew: masks would fill registers)
    static_for<U>([&](auto u) FS_INLINE {
      static_for<NT>([&](auto n) FS_INLINE { acc[u][n] = f32x4{0.f, 0.f, 0.f, 0.f}; });
      static_for<KS>([&](auto st) FS_INLINE {
        constexpr int s = decltype(st)::value, slot = s % P;
        const float up = scale_up(__builtin_amdgcn_readlane(sc, s / 2));
        u32x4 x = ring[slot];
        if (!WHOLE && s >= live) x = u32x4{0u, 0u, 0u, 0u};
        const bf16x8 w0 = widen(x[0], x[1], up), w1 = widen(x[2], x[3], up);
        static_for<NT>([&](auto n) FS_INLINE {
          acc[u][n] = mfma16(w0, hreg[s][0][n], acc[u][n]);
          acc[u][n] = mfma16(w1, hreg[s][1][n], acc[u][n]);
        });
        if constexpr (s + P < KS) ring[slot] = load(wp, s + P);
        else ring[slot] = load(wn, s + P - KS);
      });
      wp = wn;
      wn = group(nth(it * U + u + 2));
      sc = sc_next;
      sc_next = scales(nth(it * U + u + 2));
    });
    const int par = it & 1;
    static_for<U * NT>([&](auto q) FS_INLINE {
      red[((par * NW + wave) * U * NT + q) * kWave + lane] =
          acc[decltype(q)::value / NT][decltype(q)::value % NT];
    });
    __syncthreads();
    static_for<U * NT>([&](auto q) FS_INLINE {
      constexpr std::integral_constant<int, decltype(q)::value % NT> n{};
      const int g = nth(it * U + q / NT);
      if ((q + it * U) % NW == wave && g < ngroups) {
        f32x4 z = red[((par * NW + 0) * U * NT + q) * kWave + lane];
        for (int w = 1; w < NW; ++w) z += red[((par * NW + w) * U * NT + q) * kWave + lane];
        const int row0 = g * 16, b = n * 16 + li, v0 = row0 + 4 * kb;
        if constexpr (OUT == kTokenScores) {
          float zt = 0.0f;
          bool has = false;
          const bool plain =
              row0 + 16 <= a.V && __ballot(loc[n] >= row0 && loc[n] < row0 + 16) == 0;
          fold_logits<1>([&](auto) FS_INLINE { return z; }, row0, a.V, loc[n], plain, inv_t[n], m[n],
                         s_[n], zt, has);
          if (has) a.target[b] = zt;
        } else if constexpr (OUT == kSamples) {
          push_four(best[n], z, v0, a.V, static_cast<uint32_t>(a.vocab_offset + v0),
                    static_cast<uint32_t>(b), a.step, greedy[n], inv_t[n], philox);
        } else if (b < a.B) {
          // (rows may start at any element)
          const int64_t at = b * a.ld + v0;
          if constexpr (OUT == kLogitsF32) {
            typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
            float* o = static_cast<float*>(a.out) + at;
            if (v0 + 4 <= a.V) *reinterpret_cast<f32x4u*>(o) = z;
            else static_for<4>([&](auto r) FS_INLINE { if (v0 + r < a.V) o[r] = z[decltype(r)::value]; });
          } else {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
            __bf16* o = static_cast<__bf16*>(a.out) + at;
            const bf16x4 y = {static_cast<__bf16>(z[0]), static_cast<__bf16>(z[1]),
                              static_cast<__bf16>(z[2]), static_cast<__bf16>(z[3])};
            if (v0 + 4 <= a.V) *reinterpret_cast<u32x2u*>(o) = __builtin_bit_cast(u32x2u, y);
            else static_for<4>([&](auto r) FS_INLINE { if (v0 + r < a.V) o[r] = y[decltype(r)::value]; });
          }
        }
      }
    });
  }
  if constexpr (OUT == kTokenScores) {
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
  if constexpr (OUT == kSamples) {
    __shared__ float s_val[NW][NT * 16];
    __shared__ int32_t s_idx[NW][NT * 16];
    static_for<NT>([&](auto n) FS_INLINE {
      best[n].xor_reduce(16);
      best[n].xor_reduce(32);
      if (kb == 0) {
        s_val[wave][n * 16 + li] = best[n].v;
        s_idx[wave][n * 16 + li] = best[n].i;
      }
    });
    __syncthreads();
    const int c = threadIdx.x;
    if (c < NT * 16 && c < a.B) {
      ArgMax p;
      p.init();
#pragma unroll
      for (int w = 0; w < NW; ++w) p.push(s_val[w][c], s_idx[w][c]);
      const size_t o = static_cast<size_t>(c) * a.S + blockIdx.x;
      a.part_val[o] = p.v;
      a.part_idx[o] = p.i;
    }
  }
}

template <int OUT, int NT, int NW, int KS, int P, int C = 1, int U = 1, bool WHOLE = false>
hipError_t launch_fp8_shape(Fp8Args& a, hipStream_t stream) {
  if constexpr (!WHOLE)
    if (a.D == 64 * NW * KS) return launch_fp8_shape<OUT, NT, NW, KS, P, C, U, true>(a, stream);
  const auto kernel = fp8_stream_kernel<OUT, NT, NW, KS, P, WHOLE, C, U>;
  constexpr size_t smem = 2ull * NW * U * NT * kWave * sizeof(f32x4);
  static_assert(smem <= 64 * 1024, "LDS");
  static OccupancyCache cache;
  int slots = resident_blocks(kernel, NW * kWave, smem, cache);
  if (slots <= 0) return hipErrorInvalidDevice;
  slots = slots < kMaxFp8StreamBlocks ? slots : kMaxFp8StreamBlocks;
  const int clusters = (fp8_groups(a.V) + C - 1) / C;
  a.S = clusters < slots ? clusters : slots;
  kernel<<<a.S, NW * kWave, smem, stream>>>(a);
  return hipGetLastError();
}

// Waves per block, steps per wave, loads ahead, neighbouring groups per sweep and
// groups that meet at a time, by row length; 128256 rows, us.  One row of 4096: sixteen
// waves taking 128 KB (two groups) in a row that meet together 77.5, one by one 79 to 81,
// one group at a time 83.6, eight waves 79.5 to 85 (meeting in twos costs 32 rows 1 to 4,
// one row of 8192 10, and is alike elsewhere).  32 rows there: eight
// waves four loads ahead and two groups 84, one group 87.7, a whole group ahead 92,
// sixteen waves 86.  5120: five ahead 97.8, ten 100.9; 6144: sixteen waves three ahead
// 115, six 119, eight waves 119; 8192: sixteen waves four ahead 155, eight ahead (they
// spill) 176, eight waves 158 to 163.  The logits of more than 16 rows are written
// faster where a row's lines fill in one block: fp32 32 rows of 4096 by two groups 98,
// by one 103, by four 101; bf16 by four 93, two 96, one 101.  (Without the stores
// 83 to 85: their 16 MB fall on 32 pages of memory at a time.)
template <int OUT>
hipError_t launch_fp8_rows(Fp8Args& a, hipStream_t stream) {
  const int32_t D = a.D;
  if (a.B <= 16) {
    if (D <= 1024) return launch_fp8_shape<OUT, 1, 8, 2, 2>(a, stream);
    if (D <= 2048) return launch_fp8_shape<OUT, 1, 8, 4, 4>(a, stream);
    if (D <= 4096) return launch_fp8_shape<OUT, 1, 16, 4, 4, 2, 2>(a, stream);
    if (D <= 5120) return launch_fp8_shape<OUT, 1, 8, 10, 5>(a, stream);
    if (D <= 6144) return launch_fp8_shape<OUT, 1, 16, 6, 3>(a, stream);
    return launch_fp8_shape<OUT, 1, 16, 8, 4>(a, stream);
  }
  constexpr int C = OUT == kLogitsF32 ? 2 : OUT == kLogitsBf16 ? 4 : 1;
  if (D <= 1024) return launch_fp8_shape<OUT, 2, 8, 2, 2, C>(a, stream);
  if (D <= 2048) return launch_fp8_shape<OUT, 2, 8, 4, 4, C>(a, stream);
  if (D <= 4096) return launch_fp8_shape<OUT, 2, 8, 8, 4, C == 1 ? 2 : C>(a, stream);
  return launch_fp8_shape<OUT, 2, 8, 10, 5, C>(a, stream);
}

}  // namespace fs
