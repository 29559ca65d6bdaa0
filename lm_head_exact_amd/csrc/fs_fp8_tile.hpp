// fs_fp8_tile.hpp -- the 8-bit LM head for more rows than the streaming kernels
// take: a block-tiled product on the scaled 8-bit matrix instructions, and what
// its blocks make of their logits.  Instantiated in fs_fp8_tile_*.hip, which
// compile in parallel.
//
// One block computes TA vocabulary rows by TB tokens; a wave holds MR x NT tiles of
// 32 x 32 (v_mfma_scale_f32_32x32x64_f8f6f4, W as operand A; EXACT: below).  Both operands go
// through LDS, staged by direct global->LDS loads in a ring of S slots of 128 k:
// 128 bytes per row, as the 64 bf16 of the training products' slots, whose
// staging (Tile) it shares.  A slot has two steps of 64 k, whose fragments are read
// one step ahead.  32 x 32 x 64 takes half of 16 x 16 x 128's fragment registers per
// step: those of two steps and 128 accumulators fit in the 256 of a wave, two of
// which share a SIMD.
//
// Scales.  A slot is one block of 128 columns: every lane hands the instruction the
// byte of its token (B) and of its wave's vocabulary rows (A: 32 to 128 rows, within
// one block of 128).  Both live in LDS for the whole call of a block.
//
// Rounding.  The instruction aligns the products of eight neighbouring k to the
// largest of them and cuts each 13 bits below it, towards zero; sums of such groups are
// fp32 (measured: bytes planted 12 binades below the largest of their eight keep their
// first bit, two further none; those of other groups are exact).  On normal data that
// is 1.5e-5 of a logit's spread, a thousandth of what the values' own four bits leave.
// Where the products of a logit share a sign (h along the row of W) nothing averages
// it: such a logit comes out 1e-5 of it too small (7e-4 of 82, D = 1024 or 4096).
// Exact products (EXACT) widen the same fragments to bf16, which holds four bits times a
// power of two: four products of 16 k for one of 64, at half its rate.  Samples, logits in
// fp32 and scores on few entries or of few rows take them (fs_fp8_tile_*.hip).
#pragma once

#include "fs_fp8.hpp"
#include "fs_sampler.hpp"

namespace fs {

typedef int i32x8 __attribute__((ext_vector_type(8)));

template <int WA_, int WB_, int MR_, int NT_, int S_>
struct Fp8Tile : Tile<kFrag, kKC, WA_, WB_, 2 * MR_, 2 * NT_, S_, 64, false, true> {
  using Base = Tile<kFrag, kKC, WA_, WB_, 2 * MR_, 2 * NT_, S_, 64, false, true>;
  static constexpr int WA = WA_, WB = WB_, MR = MR_, NT = NT_, S = S_;
  static constexpr int TA = Base::TA, TB = Base::TB, NW = Base::NW;
  static_assert(128 % (32 * MR) == 0, "a wave's rows lie in one block of scales");
  static constexpr int kVB = (TA + kQuantBlock - 1) / kQuantBlock;  // blocks of rows in a tile
  using Base::IA;
  using Base::IB;
  using Base::kStage;
  using Base::kStageA;

  // LDS (fp8_lds): the ring, the tokens' scales [KB][TB], the rows' [kVB][KB].

  // Fragment f (32 rows) of step s of the staged tile at `buf`: lane (li, kb) gets row
  // li and bytes 64 s + 32 kb + 0..31.
  __device__ __forceinline__ static i32x8 frag_w(const unsigned char* buf, int f, int s) {
    const int lane = threadIdx.x & (kWave - 1), li = lane & 31, kb = lane >> 5;
    const unsigned char* a =
        buf + ((2 * f + (li >> 4)) * 2 + s) * 1024 + (2 * kb * 16 + (li & 15)) * 16;
    return join(a, a + 256);
  }
  __device__ __forceinline__ static i32x8 frag_h(const unsigned char* buf, int f, int s) {
    const int lane = threadIdx.x & (kWave - 1), li = lane & 31, kb = lane >> 5;
    const unsigned char* a = buf + (f * 32 + li) * 128;
    const int piece = 4 * s + 2 * kb, x = Base::kc_swizzle(li);
    return join(a + ((piece ^ x) * 16), a + (((piece + 1) ^ x) * 16));
  }
  __device__ __forceinline__ static i32x8 join(const unsigned char* a, const unsigned char* b) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(a), y = *reinterpret_cast<const u32x4*>(b);
    return __builtin_bit_cast(i32x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  }

  // acc[m][n] of tokens b0 + wave_b() + 32 n + (lane mod 32), vocabulary rows a0 +
  // wave_a() + 32 m + 8 q + 4 (lane / 32) + r in element 4 q + r.  LDS is free for
  // reuse when it returns.  The loop is the training products': one barrier per slot,
  // before its last step's products, behind which the slot S ahead is staged.
  // EXACT: by bf16 products of the widened bytes.
  template <bool EXACT>
  __device__ __forceinline__ static void run(const Fp8Args& a, int a0, int b0,
                                             f32x16 (&acc)[MR][NT], unsigned char* smem) {
    static_for<MR>([&](auto m) FS_INLINE {
      static_for<NT>([&](auto n) FS_INLINE { acc[m][n] = f32x16{}; });
    });
    // bf16 units: two bytes
    const Operand w = {reinterpret_cast<const __bf16*>(a.w), 8ll * a.D, (a.V - 1) / 16 + 1, a.D / 2};
    const Operand h = {reinterpret_cast<const __bf16*>(a.hq), a.Dp / 2, a.B, a.Dp / 2};
    const int lane = threadIdx.x & (kWave - 1);
    const int KB = a.KB, nk = KB;
    unsigned char* s_h = smem + Base::kSmemBytes;
    unsigned char* s_w = s_h + KB * TB;
    for (int i = threadIdx.x; i < KB * (TB / 4); i += Base::kThreads) {
      const int kt = i / (TB / 4), c = i % (TB / 4) * 4;
      // (rows of hscale are Bp long, a multiple of 256, and b0 + TB is at most Bp)
      *reinterpret_cast<uint32_t*>(s_h + kt * TB + c) =
          *reinterpret_cast<const uint32_t*>(a.hscale + static_cast<size_t>(kt) * a.Bp + b0 + c);
    }
    const int vblocks = quant_blocks(a.V);
    for (int i = threadIdx.x; i < kVB * KB; i += Base::kThreads) {
      const int vb = min(a0 / kQuantBlock + i / KB, vblocks - 1);
      s_w[i] = a.wscale[static_cast<size_t>(vb) * KB + i % KB];
    }
    __syncthreads();
    const unsigned char* my_h = s_h + Base::wave_b() + (lane & 31);
    const unsigned char* my_w =
        s_w + ((a0 % kQuantBlock + Base::wave_a()) / kQuantBlock) * KB;

    typename Base::template Stager<kFrag, TA, IA> sa;
    typename Base::template Stager<kKC, TB, IB> sb;
    sa.init(w, a0);
    sb.init(h, b0);
    const int ragged = w.k / 64;  // (h is padded to whole blocks)
    auto stage = [&](int kt, unsigned char* dst) FS_INLINE {
      sa.stage(kt, dst);
      sb.stage(kt, dst + kStageA);
    };
    auto prepare = [&](int kt) FS_INLINE {
      if (kt == ragged) sa.offsets(w, a0, w.k - kt * 64);
    };
    const int fa = Base::wave_a() / 32, fb = Base::wave_b() / 32;
    i32x8 fw[2][MR], fh[2][NT];
    int sw[2], sh[2][NT];  // scales of the slot being multiplied and of the next one
    auto read = [&](auto set, auto step, const unsigned char* tile) FS_INLINE {
      constexpr int x = decltype(set)::value, s = decltype(step)::value;
      static_for<NT>([&](auto n) FS_INLINE { fh[x][n] = frag_h(tile + kStageA, fb + n, s); });
      static_for<MR>([&](auto m) FS_INLINE { fw[x][m] = frag_w(tile, fa + m, s); });
    };
    auto read_scales = [&](int kt, int x) FS_INLINE {
      sw[x] = my_w[kt];
      static_for<NT>([&](auto n) FS_INLINE { sh[x][n] = my_h[kt * TB + 32 * static_cast<int>(n)]; });
    };
    auto mma = [&](auto set) FS_INLINE {
      constexpr int x = decltype(set)::value;
      if constexpr (EXACT) {
        // 16 k at a time: eight of each half's 32, in both operands alike
        static_for<4>([&](auto i) FS_INLINE {
          constexpr int j = 2 * decltype(i)::value;
          bf16x8 h[NT];
          static_for<NT>([&](auto n) FS_INLINE {
            h[n] = widen(fh[x][n][j], fh[x][n][j + 1], scale_up(sh[0][n]));
          });
          static_for<MR>([&](auto m) FS_INLINE {
            const bf16x8 w = widen(fw[x][m][j], fw[x][m][j + 1], scale_up(sw[0]));
            static_for<NT>([&](auto n) FS_INLINE {
              acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, h[n], acc[m][n], 0, 0, 0);
            });
          });
        });
        return;
      }
      static_for<MR>([&](auto m) FS_INLINE {
        static_for<NT>([&](auto n) FS_INLINE {
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fw[x][m], fh[x][n], acc[m][n], 0, 0, 0, sw[0], 0, sh[0][n]);
        });
      });
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    prepare(0);
    stage(0, smem);
    __builtin_amdgcn_sched_barrier(0);
    [&](const unsigned char* __restrict__ from, unsigned char* __restrict__ to) FS_INLINE {
      static_for<S - 1>([&](auto i) FS_INLINE {
        const int kt = min(1 + static_cast<int>(i), nk - 1);
        prepare(kt);
        stage(kt, to + i * kStage);
        __builtin_amdgcn_sched_barrier(0);
      });
      Base::template wait_lgkm0_vm<(S - 1) * (IA + IB)>();
      Base::barrier();
      read_scales(0, 0);
      read(I0{}, I0{}, from);
      read(I1{}, I1{}, from);
      mma(I0{});
      if constexpr (!EXACT) interleave<0>();
      __builtin_amdgcn_sched_barrier(0);
    }(smem, smem + kStage);
    int slot = 0;
    for (int kt = 0; kt + 1 < nk; ++kt) {
      const int next = slot == S - 1 ? 0 : slot + 1;
      const int ahead = min(kt + S, nk - 1);
      prepare(ahead);
      __builtin_amdgcn_sched_barrier(0);
      Base::template wait_lgkm0_vm<(S - 2) * (IA + IB)>();
      Base::barrier();
      [&](const unsigned char* __restrict__ from, unsigned char* __restrict__ to) FS_INLINE {
        read_scales(kt + 1, 1);
        read(I0{}, I0{}, from);
        stage(ahead, to);
        mma(I1{});
        if constexpr (!EXACT) interleave<IA + IB>();
        __builtin_amdgcn_sched_barrier(0);
        sw[0] = sw[1];
        static_for<NT>([&](auto n) FS_INLINE { sh[0][n] = sh[1][n]; });
        read(I1{}, I1{}, from);
        mma(I0{});
        if constexpr (!EXACT) interleave<0>();
        __builtin_amdgcn_sched_barrier(0);
      }(smem + next * kStage, smem + slot * kStage);
      slot = next;
    }
    mma(I1{});
    Base::template wait_lgkm0_vm<0>();  // the trailing (clamped) loads land before LDS is reused
    Base::barrier();
  }

  // One step's products with the LDS reads of the next step and `loads` direct loads
  // spread between them.
  template <int loads>
  __device__ __forceinline__ static void interleave() {
    constexpr int kMfma = MR * NT, kReads = 2 * (MR + NT), kSlots = kReads + loads;
    static_for<kSlots>([&](auto i) FS_INLINE {
      constexpr int k = decltype(i)::value;
      constexpr int from = kMfma * k / kSlots, to = kMfma * (k + 1) / kSlots;
      if constexpr (k < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      else __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      if constexpr (to > from) __builtin_amdgcn_sched_group_barrier(0x008, to - from, 0);
    });
  }
};

template <class T, int OUT, bool EXACT>
__global__ __launch_bounds__(T::kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void fp8_tile_kernel(Fp8Args a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn_smem[];
  int tile, btile;
  if (!xcd_tile<4>(blockIdx.x, a.S, (a.B + T::TB - 1) / T::TB, tile, btile)) return;
  const int a0 = tile * T::TA, b0 = btile * T::TB;
  f32x16 acc[T::MR][T::NT];
  T::template run<EXACT>(a, a0, b0, acc, dyn_smem);

  const int lane = threadIdx.x & (kWave - 1), li = lane & 31, kb = lane >> 5;
  const int row0 = a0 + T::wave_a(), col0 = b0 + T::wave_b();
  constexpr int kQuads = 4 * T::MR;
  // A wave's logits of one token, in quads of four consecutive vocabulary rows: quad i
  // has rows 8 i + 4 kb of the wave's.
  auto quad = [&](auto i, auto n) FS_INLINE {
    constexpr int m = decltype(i)::value / 4, q = decltype(i)::value % 4;
    const f32x16 x = acc[m][decltype(n)::value];
    return f32x4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
  };

  if constexpr (OUT == kLogitsBf16 || OUT == kLogitsF32) {
    // Through LDS, so that a store covers whole stretches of a token's row: a wave's
    // 32 tokens at a time (of fp32 16, which is what LDS holds), each wave in a region
    // of its own.
    constexpr int kSize = OUT == kLogitsF32 ? 4 : 2;
    constexpr int kTokens = OUT == kLogitsF32 ? 16 : 32;
    constexpr int kCols = 32 * T::MR, kPitch = kCols * kSize + 16;
    static_assert(static_cast<size_t>(T::NW) * kTokens * kPitch <= T::kSmemBytes, "LDS");
    unsigned char* mine = dyn_smem + T::wave() * (kTokens * kPitch);
    static_for<T::NT * 32 / kTokens>([&](auto part) FS_INLINE {
      constexpr int n = decltype(part)::value * kTokens / 32;
      constexpr int first = decltype(part)::value * kTokens % 32;  // token of the 32
      if (li >= first && li < first + kTokens) {
        static_for<kQuads>([&](auto i) FS_INLINE {
          const f32x4 z = quad(i, std::integral_constant<int, n>{});
          unsigned char* p = mine + (li - first) * kPitch + (8 * static_cast<int>(i) + 4 * kb) * kSize;
          if constexpr (OUT == kLogitsF32) {
            *reinterpret_cast<f32x4*>(p) = z;
          } else {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<bf16x4*>(p) =
                bf16x4{static_cast<__bf16>(z[0]), static_cast<__bf16>(z[1]),
                       static_cast<__bf16>(z[2]), static_cast<__bf16>(z[3])};
          }
        });
      }
      __builtin_amdgcn_wave_barrier();  // (the wave's own LDS operations complete in order)
      constexpr int kPer = 16 / kSize;       // elements of 16 bytes
      constexpr int kLanes = kCols / kPer;   // lanes per token
      constexpr int kRows = kWave / kLanes;  // tokens per store
      const int token0 = col0 + 32 * n + first;
      // Rows may start at any element: the stores are of 16 bytes all the same.  Past the
      // caches only where every row starts a line (5607 rows of 77144 bf16: 291 us through
      // them, 422 past them).
      typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
      if (row0 + kCols <= a.V) {
        static_for<kTokens / kRows>([&](auto i) FS_INLINE {
          const int r = static_cast<int>(i) * kRows + lane / kLanes, c = lane % kLanes;
          const u32x4 v = *reinterpret_cast<const u32x4*>(mine + r * kPitch + c * 16);
          unsigned char* o = static_cast<unsigned char*>(a.out) +
                             ((token0 + r) * a.ld + row0 + c * kPer) * kSize;
          if (token0 + r >= a.B) return;
          if (a.lines) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(o));
          else *reinterpret_cast<u32x4u*>(o) = v;
        });
      } else {  // the end of the vocabulary: one element per lane
        for (int i = lane; i < kTokens * kCols; i += kWave) {
          const int r = i / kCols, c = i % kCols;
          if (token0 + r < a.B && row0 + c < a.V) {
            const int64_t at = (token0 + r) * a.ld + row0 + c;
            if constexpr (OUT == kLogitsF32)
              static_cast<float*>(a.out)[at] = *reinterpret_cast<const float*>(mine + r * kPitch + c * 4);
            else
              static_cast<uint16_t*>(a.out)[at] =
                  *reinterpret_cast<const uint16_t*>(mine + r * kPitch + c * 2);
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    });
  }

  if constexpr (OUT == kTokenScores) {
    float2* red = reinterpret_cast<float2*>(dyn_smem);  // [WA][TB]
    const bool inside = row0 + 32 * T::MR <= a.V;
    static_for<T::NT>([&](auto n) FS_INLINE {
      const int b = col0 + 32 * static_cast<int>(n) + li, bc = min(b, a.B - 1);
      const float inv_t = score_inv_t(a.temperature, bc);
      const int loc = target_row(a.ids[bc], a.vocab_offset, a.V);
      const bool hit = loc >= row0 && loc < row0 + 32 * T::MR;
      const bool plain = inside && __ballot(hit) == 0;
      float m = LseAcc::kMasked, s = 0.0f, zt = 0.0f;
      bool has = false;
      fold_logits<kQuads, 8>([&](auto i) FS_INLINE { return quad(i, n); }, row0, a.V, loc, plain,
                             inv_t, m, s, zt, has);
      pair_xor(m, s, 32);  // (the target's own logit is made apart, exactly)
      if (kb == 0) red[(T::wave() / T::WB) * T::TB + T::wave_b() + 32 * n + li] = float2{m, s};
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

  if constexpr (OUT == kSamples) {
    float2* red = reinterpret_cast<float2*>(dyn_smem);  // [WA][TB]: value, id
    const Philox philox(a.seed);
    static_for<T::NT>([&](auto n) FS_INLINE {
      const int b = col0 + 32 * static_cast<int>(n) + li;
      const float temp = a.temperature[min(b, a.B - 1)];
      const bool greedy = row_is_greedy(temp);
      const float inv_t = row_inv_temperature(temp);
      ArgMax best;
      best.init();
      static_for<kQuads>([&](auto i) FS_INLINE {
        const int v0 = row0 + 8 * static_cast<int>(i) + 4 * kb;
        push_four(best, quad(i, n), v0, a.V, static_cast<uint32_t>(a.vocab_offset + v0),
                  static_cast<uint32_t>(b), a.step, greedy, inv_t, philox);
      });
      best.xor_reduce(32);
      if (kb == 0)
        red[(T::wave() / T::WB) * T::TB + T::wave_b() + 32 * n + li] =
            float2{best.v, __int_as_float(best.i)};
    });
    __syncthreads();
    for (int c = threadIdx.x; c < T::TB; c += T::kThreads) {
      if (b0 + c >= a.B) break;
      ArgMax p;
      p.init();
#pragma unroll
      for (int w = 0; w < T::WA; ++w) {
        const float2 o = red[w * T::TB + c];
        p.push(o.x, __float_as_int(o.y));
      }
      const size_t o = static_cast<size_t>(b0 + c) * a.S + tile;
      a.part_val[o] = p.v;
      a.part_idx[o] = p.i;
    }
  }
}

// ---- the tiles of kFp8TileShapes ----
using Fp8Tall64 = Fp8Tile<8, 1, 1, 2, 3>;
using Fp8Tall128 = Fp8Tile<4, 2, 2, 2, 3>;
using Fp8Tall256 = Fp8Tile<2, 4, 4, 2, 2>;
using Fp8Short64 = Fp8Tile<2, 2, 1, 1, 3>;
using Fp8Short256 = Fp8Tile<2, 2, 2, 2, 2>;

template <class T, int SHAPE, int OUT, bool EXACT>
hipError_t launch_fp8_tile(Fp8Args& a, hipStream_t stream) {
  constexpr Fp8TileShape c = kFp8TileShapes[SHAPE];
  static_assert(T::TA == c.rows && T::TB == c.tokens && T::S == c.slots, "the shape of the rule");
  static_assert(T::kThreads == (T::TA == kTallRows ? 512 : 256), "threads_of");
  a.S = static_cast<int32_t>((static_cast<int64_t>(a.V) + T::TA - 1) / T::TA);
  static SmemRaised raised;
  const hipError_t e = raise_smem(&fp8_tile_kernel<T, OUT, EXACT>, kFp8Lds, raised);
  if (e != hipSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(a.S) * ((a.B + T::TB - 1) / T::TB);
  fp8_tile_kernel<T, OUT, EXACT><<<static_cast<unsigned>((tiles + 7) / 8 * 8), T::kThreads,
                            fp8_lds(c, a.D), stream>>>(a);
  return hipGetLastError();
}

template <int OUT, bool EXACT = false>
hipError_t launch_fp8_tiles(Fp8Args& a, hipStream_t stream) {
  switch (fp8_tile(a.B, a.D, a.V)) {
    case LogitsTile::kTall64: return launch_fp8_tile<Fp8Tall64, 0, OUT, EXACT>(a, stream);
    case LogitsTile::kTall128: return launch_fp8_tile<Fp8Tall128, 1, OUT, EXACT>(a, stream);
    case LogitsTile::kTall256: return launch_fp8_tile<Fp8Tall256, 2, OUT, EXACT>(a, stream);
    case LogitsTile::kShort64: return launch_fp8_tile<Fp8Short64, 3, OUT, EXACT>(a, stream);
    default: return launch_fp8_tile<Fp8Short256, 4, OUT, EXACT>(a, stream);
  }
}

}  // namespace fs
