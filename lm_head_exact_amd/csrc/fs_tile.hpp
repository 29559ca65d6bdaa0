// fs_tile.hpp -- the block-tiled bf16 matrix product of the training operators
// on gfx950: C[b][a] = sum_k A(a, k) B(b, k), fp32 accumulators.
//
// One block of 8 waves (two per SIMD, one block per CU), or of 4 waves where a
// grid of those would leave CUs idle, computes TA x TB elements of C; a wave
// holds MR x NT tiles of 16 x 16 (v_mfma_f32_16x16x32_bf16, A as the MFMA's
// rows).  Both operands go through LDS, staged by direct global->LDS loads in a
// ring of S slots of BK = 64 or 32 k.  (64 halves the barriers; an operand read
// by transposing takes 32, whose finer slots hold the same bytes in flight with
// one k step of registers fewer.)  An operand is either
//   K-contiguous (KC)  element (i, k) at p[i * pitch + k]: 16-byte pieces
//                      along k, read back as they are (ds_read_b128);
//   K-major (KM)       element (i, k) at p[k * pitch + i]: 16-byte pieces
//                      along i; the transposing LDS read
//                      (ds_read_b64_tr_b16) hands every lane its k's, so no
//                      operand is ever transposed in memory.
//   fragment order     W as fs_pack_weights stores it (groups of 16 rows, one
//                      contiguous KB per group and 32 k): staged and read as
//                      it is (ds_read_b128, lanes in order).
// The three products of the LM head are (KC or fragment order, KC) for logits,
// (KM, KC) for the gradient of the hidden states and (KM, KM) for the gradient
// of W.
//
// LDS layouts.  KC: rows of 64 k (128 bytes, 8 pieces), piece j of row i at
// slot j ^ (i mod 8); rows of 32 k (4 pieces) at slot j ^ (i / 2 mod 4): the 16
// rows of a read cover the banks evenly.  KM: rows of one k (T elements), the 32-byte unit u of
// row k at unit u ^ g(k), g(k) = (k mod 4) + 4 (k / 8 mod 2): a transposing
// read takes from each of its four 16-lane groups four rows of one unit; g
// spreads the eight rows of 32 lanes over the eight 32-byte bank groups.  The
// direct loads write LDS in lane order, so the permutation is applied to the
// addresses they read.
//
// Bounds.  Rows and columns past an operand's end are read at its last one, and
// so are the k's of a KM operand; the k's past a KC or fragment-order operand's
// end are offsets beyond the buffer's size, which load zeros: no access leaves
// the operand.  What lies past the end is masked by the epilogue (rows of A and
// B) or multiplied by the other operand's zeros (k).  (Where A's k's end is
// ragged it is W of the logits, and an infinite entry of it read again would
// make inf * 0 of those zeros.)
#pragma once

#include "fs_mma.hpp"

namespace fs {

enum Layout { kKC = 0, kKM = 1, kFrag = 2 };

struct Operand {
  const __bf16* p;
  int64_t pitch;  // elements: between rows (KC), between k's (KM), between groups (fragment order)
  int32_t n;      // rows (KM: a multiple of 8); fragment order: groups of 16 rows
  int32_t k;      // k's; KC: a multiple of 8; fragment order: a multiple of 32
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int LA_, int LB_, int WA_, int WB_, int MR_, int NT_, int S_, int BK_ = 64,
          bool NTA_ = false, bool ROWS32_ = false>
struct Tile {
  static constexpr int LA = LA_, LB = LB_;
  static_assert(LB != kFrag, "W is operand A");
  static constexpr int WA = WA_, WB = WB_, MR = MR_, NT = NT_, S = S_;
  static constexpr int NW = WA * WB;
  static constexpr int kThreads = NW * kWave;
  static constexpr int TA = WA * MR * 16, TB = WB * NT * 16;
  static constexpr int BK = BK_;  // k's of a ring slot: 64 or 32
  // A is read once and by one block: its loads carry the non-temporal hint
  static constexpr bool NTA = NTA_;
  static constexpr int KS = BK / 32;
  static constexpr int kStageA = TA * BK * 2, kStageB = TB * BK * 2;  // bytes
  static constexpr int kStage = kStageA + kStageB;
  static constexpr size_t kSmemBytes = static_cast<size_t>(S) * kStage;
  static constexpr int IA = kStageA / (NW * 1024), IB = kStageB / (NW * 1024);
  static_assert(kStageA % (NW * 1024) == 0 && kStageB % (NW * 1024) == 0, "staging divides evenly");
  static_assert((LA != kKM || TA % 128 == 0) && (LB != kKM || TB % 128 == 0),
                "KM swizzle needs 8 units a row");
  static_assert(kSmemBytes <= 160 * 1024, "LDS");
  static constexpr int kBufferFlags = 0x00020000;
  // The buffers' size in bytes, above every offset of an operand's; and an offset
  // past it, for which a load gives zeros.
  static constexpr int kBufferBytes = 0x7FFFFFFF;
  static constexpr int kPastEnd = static_cast<int>(0x80000000u);

  __device__ __forceinline__ static int wave() {
    return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  }
  // First row of A and of B that this wave's accumulators cover, in the tile.
  __device__ __forceinline__ static int wave_a() { return (wave() / WB) * MR * 16; }
  __device__ __forceinline__ static int wave_b() { return (wave() % WB) * NT * 16; }

  template <int N>
  __device__ __forceinline__ static void wait_vm() {
    static_assert(N >= 0 && N <= 63, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  }
  // Workgroup barrier without the fence of __syncthreads (which would wait
  // for every load in flight); the callers wait for what they need.
  __device__ __forceinline__ static void barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  // The permutation of 16-byte pieces in a KC row.
  // (ROWS32: for reads of 32 rows, 16 lanes of which go together: rows of which two
  // are alike modulo 8, one of each two from 16 on.)
  __device__ __forceinline__ static int kc_swizzle(int r) {
    return BK != 64 ? (r >> 1) & 3 : ROWS32_ ? (r & 7) ^ ((r >> 4) & 1) : r & 7;
  }
  // The permutation of 32-byte units in a KM row.
  __device__ __forceinline__ static int km_swizzle(int k) { return (k & 3) | ((k >> 1) & 4); }

  // Staging of one operand: byte offsets, from the first element of a k tile of
  // the operand's rows i0 .., of the pieces this lane loads.  They are the same
  // for every k tile (the tile's start is in scalar registers) but the last,
  // ragged one.
  template <int L, int T, int I, bool NT_LOADS = false>
  struct Stager {
    const __bf16* base;  // rows i0 .. at k = 0
    int64_t step;        // elements from one k tile to the next
    int off[I];
    __device__ __forceinline__ void init(const Operand& o, int i0) {
      base = o.p + (L == kKM ? static_cast<int64_t>(i0) : (L == kFrag ? i0 / 16 : i0) * o.pitch);
      step = L == kKM ? BK * o.pitch : L == kFrag ? BK * 16 : BK;
      offsets(o, i0, BK);
    }
    // Offsets for a k tile of `ks` k's.
    __device__ __forceinline__ void offsets(const Operand& o, int i0, int ks) {
      const int lane = threadIdx.x & (kWave - 1);
      static_for<I>([&](auto i) FS_INLINE {
        const int q = (wave() * I + static_cast<int>(i)) * kWave + lane;  // 16-byte slot
        if constexpr (L == kKM) {
          constexpr int P = T / 8;  // pieces per row of one k
          const int k = q / P, piece = (q % P) ^ (km_swizzle(k) << 1);
          off[i] = min(piece * 8, o.n - 8 - i0) * 2 + min(k, ks - 1) * static_cast<int>(o.pitch * 2);
        } else if constexpr (L == kFrag) {  // pieces (group, k step of the tile) of 1 KB
          const int piece = q / kWave;
          off[i] = piece % KS * 32 < ks
                       ? static_cast<int>(min(piece / KS, o.n - 1 - i0 / 16) * o.pitch) * 2 +
                             lane * 16 + piece % KS * 1024
                       : kPastEnd;
        } else {
          constexpr int P = BK / 8;  // pieces per row
          const int r = q / P, piece = (q % P) ^ kc_swizzle(r);
          off[i] = piece * 8 < ks
                       ? (static_cast<int>(min(r, o.n - 1 - i0) * o.pitch) + piece * 8) * 2
                       : kPastEnd;
        }
      });
    }
    // Tile kt into LDS at `dst`.
    __device__ __forceinline__ void stage(int kt, unsigned char* dst) const {
      const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<__bf16*>(base + kt * step), 0, kBufferBytes, kBufferFlags);
      static_for<I>([&](auto i) FS_INLINE {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc,
            (__attribute__((address_space(3))) void*)(dst + (wave() * I + static_cast<int>(i)) * 1024),
            16, off[i], 0, 0, NT_LOADS ? 2 : 0);
      });
    }
  };

  // Fragment f (16 rows from f * 16 of the staged tile) of k step s of the
  // operand at `buf`: lane (li, kb) gets row li, k = 32 s + 8 kb + 0..7.
  template <int L, int T>
  __device__ __forceinline__ static bf16x8 frag(const unsigned char* buf, int f, int s) {
    const int lane = threadIdx.x & (kWave - 1);
    if constexpr (L == kKM) {
      const int g = lane >> 4, i = lane & 15;
      // row k = 32 s + 8 g + 4 half + i / 4: its swizzle does not depend on s or half
      const int c = (i >> 2) | ((g & 1) << 2);
      const unsigned char* a =
          buf + (8 * g + (i >> 2)) * (T * 2) + ((f ^ c) * 32 + (i & 3) * 8) + s * 32 * (T * 2);
      const s16x4 lo = tr(a), hi = tr(a + 4 * (T * 2));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else if constexpr (L == kFrag) {
      return __builtin_bit_cast(
          bf16x8, *reinterpret_cast<const u32x4*>(buf + (f * KS + s) * 1024 + lane * 16));
    } else {
      const int li = lane & 15, kb = lane >> 4;
      const unsigned char* a =
          buf + (f * 16 + li) * (BK * 2) + (((s * 4 + kb) ^ kc_swizzle(li)) * 16);
      return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(a));
    }
  }
  __device__ __forceinline__ static s16x4 tr(const unsigned char* a) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(const_cast<unsigned char*>(a)));
  }

  // acc[m][n] of C rows b0 + wave_b() + 16 n + li, columns a0 + wave_a() + 16 m
  // + 4 kb + 0..3, over k tiles [kt0, kt1).  LDS is free for reuse when it
  // returns.
  //
  // Every k step's fragments are read from LDS one step ahead, into the other
  // of two register sets, while the MFMAs of the current step run.  A k tile
  // has one barrier, before its last step's MFMAs: there each wave has read the
  // whole of the tile (its slot may be refilled) and waited for its share of
  // the next one (which may then be read).  The direct loads of tile kt + S
  // go out right behind that barrier and have S - 1 tiles of time to land.
  // 4096 x 4096 x 128256 in any of the three pairs of layouts: 1.25 to 1.3
  // PFLOP/s.  Under it the clock falls from 2.4 GHz to 1.8 or 1.9, as under every
  // product that draws the board's 1400 W, with the matrix cores busy 62 to 70%
  // of its cycles.  Of copies that skip one part each, the one without
  // the direct loads runs at 1.6, without the LDS reads at 1.35, without both
  // at 1.8 PFLOP/s; with every load an L2 hit it is 1.38.
  __device__ __forceinline__ static void run(const Operand& A, const Operand& B, int a0, int b0,
                                             int kt0, int kt1, f32x4 (&acc)[MR][NT],
                                             unsigned char* smem) {
    zero_acc(acc);
    Stager<LA, TA, IA, NTA> sa;
    Stager<LB, TB, IB> sb;
    sa.init(A, a0);
    sb.init(B, b0);
    // the first k tile that is not whole for an operand
    const int raggedA = A.k / BK, raggedB = B.k / BK;
    auto stage = [&](int kt, unsigned char* dst) FS_INLINE {
      sa.stage(kt, dst);
      sb.stage(kt, dst + kStageA);
    };
    // k tiles past the last are staged as the last one again (never used)
    auto prepare = [&](int kt) FS_INLINE {
      if (kt == raggedA) sa.offsets(A, a0, A.k - kt * BK);
      if (kt == raggedB) sb.offsets(B, b0, B.k - kt * BK);
    };
    const int fa = wave_a() / 16, fb = wave_b() / 16;
    bf16x8 a[2][MR], b[2][NT];
    // k step s of a staged tile into register set `set`
    auto read = [&](auto set, auto s, const unsigned char* tile) FS_INLINE {
      constexpr int x = decltype(set)::value, ks = decltype(s)::value;
      static_for<NT>([&](auto n) FS_INLINE { b[x][n] = frag<LB, TB>(tile + kStageA, fb + n, ks); });
      static_for<MR>([&](auto m) FS_INLINE { a[x][m] = frag<LA, TA>(tile, fa + m, ks); });
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    // A tile is read while others are loaded into other slots: the qualifiers
    // below say so (without them the compiler would let no transposing read
    // pass a direct load).
    prepare(kt0);
    stage(kt0, smem);
    __builtin_amdgcn_sched_barrier(0);
    [&](const unsigned char* __restrict__ from, unsigned char* __restrict__ to) FS_INLINE {
      static_for<S - 1>([&](auto i) FS_INLINE {
        const int kt = min(kt0 + 1 + static_cast<int>(i), kt1 - 1);
        prepare(kt);
        stage(kt, to + i * kStage);
        __builtin_amdgcn_sched_barrier(0);
      });
      wait_lgkm0_vm<(S - 1) * (IA + IB)>();
      barrier();
      read(I0{}, I0{}, from);
      if constexpr (KS == 2) {
        read(I1{}, I1{}, from);
        mma_step(a[0], b[0], acc);
        interleave<0>();
        __builtin_amdgcn_sched_barrier(0);
      }
    }(smem, smem + kStage);
    int slot = 0;
    // From the last step of tile kt, whose fragments are in set X, to the next
    // tile: the barrier, the next tile's first fragments into the other set, the
    // loads of the tile S ahead and the step's MFMAs; with two steps per tile
    // also the next tile's first step and the reads of its second.
    auto advance = [&](auto set, int kt) FS_INLINE {
      constexpr int x = decltype(set)::value;
      const int next = slot == S - 1 ? 0 : slot + 1;
      const int ahead = min(kt + S, kt1 - 1);
      prepare(ahead);
      __builtin_amdgcn_sched_barrier(0);
      wait_lgkm0_vm<(S - 2) * (IA + IB)>();
      barrier();
      [&](const unsigned char* __restrict__ from, unsigned char* __restrict__ to) FS_INLINE {
        read(std::integral_constant<int, 1 - x>{}, I0{}, from);
        stage(ahead, to);
        mma_step(a[x], b[x], acc);
        interleave<IA + IB>();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (KS == 2) {
          read(I1{}, I1{}, from);
          mma_step(a[0], b[0], acc);
          interleave<0>();
          __builtin_amdgcn_sched_barrier(0);
        }
      }(smem + next * kStage, smem + slot * kStage);
      slot = next;
    };
    if constexpr (KS == 2) {
      for (int kt = kt0; kt + 1 < kt1; ++kt) advance(I1{}, kt);
      mma_step(a[1], b[1], acc);
    } else {
      // (the last tile advances too, to one that is staged but not used: an
      // ending of its own for either set would cost registers)
      int kt = kt0;
      for (; kt + 1 < kt1; kt += 2) {
        advance(I0{}, kt);
        advance(I1{}, kt + 1);
      }
      if (kt < kt1) advance(I0{}, kt);
    }
    wait_lgkm0_vm<0>();  // the trailing (clamped) loads land before LDS is reused
    barrier();
  }

  // Writes the wave's part of C as bf16 rows of its columns, through LDS, so
  // that each store covers whole stretches of rows with 16 bytes per lane (as
  // the accumulators lie, a store would be 8 bytes per lane in stretches of
  // 32).  value(m, n): the four columns of accumulator (m, n), packed.
  // keep(r, c): whether the eight columns from c of row r are written, to
  // out(r) + c elements (r and c in the wave's part).  Each wave has a region
  // of its own: no barrier.
  template <bool NTS = false, class Value, class Out, class Keep>
  __device__ __forceinline__ static void store_rows(unsigned char* smem, Value value, Out out,
                                                    Keep keep) {
    constexpr int kPitch = MR * 32 + 16;  // bytes of a row: its columns and a shift of 4 banks
    constexpr int HN = NT > 4 ? 4 : NT > 1 ? NT / 2 : 1;  // tiles of 16 rows at a time
    static_assert(NT % HN == 0, "rounds");
    static_assert(static_cast<size_t>(NW) * HN * 16 * kPitch <= kSmemBytes, "LDS");
    const int lane = threadIdx.x & (kWave - 1), li = lane & 15, kb = lane >> 4;
    unsigned char* mine = smem + wave() * (HN * 16 * kPitch);
    constexpr int kLanes = MR * 2;  // lanes per row, 16 bytes each
    constexpr int kRows = kWave / kLanes;
    static_for<NT / HN>([&](auto h) FS_INLINE {
      static_for<HN>([&](auto n) FS_INLINE {
        static_for<MR>([&](auto m) FS_INLINE {
          *reinterpret_cast<uint64_t*>(mine + (16 * n + li) * kPitch + m * 32 + kb * 8) =
              value(m, std::integral_constant<int, decltype(h)::value * HN + decltype(n)::value>{});
        });
      });
      static_for<HN * 16 / kRows>([&](auto i) FS_INLINE {
        const int r = static_cast<int>(i) * kRows + lane / kLanes, c = (lane % kLanes) * 8;
        const u32x4 v = *reinterpret_cast<const u32x4*>(mine + r * kPitch + c * 2);
        const int row = static_cast<int>(h) * HN * 16 + r;
        if (keep(row, c)) {
          u32x4* p = reinterpret_cast<u32x4*>(out(row) + c);
          if constexpr (NTS) __builtin_nontemporal_store(v, p);
          else *p = v;
        }
      });
    });
  }

  // LDS reads of one k step's fragments.
  static constexpr int kReads = MR * (LA == kKM ? 2 : 1) + NT * (LB == kKM ? 2 : 1);
  // The order of one step: its MFMAs with the LDS reads of the next step, and
  // `loads` direct loads, spread between them.
  template <int loads>
  __device__ __forceinline__ static void interleave() {
    constexpr int kMfma = MR * NT;
    constexpr int kSlots = kReads + loads;
    static_for<kSlots>([&](auto i) FS_INLINE {
      constexpr int k = decltype(i)::value;
      constexpr int from = kMfma * k / kSlots, to = kMfma * (k + 1) / kSlots;
      if constexpr (k < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      else __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      if constexpr (to > from) __builtin_amdgcn_sched_group_barrier(0x008, to - from, 0);
    });
  }

  template <int N>
  __device__ __forceinline__ static void wait_lgkm0_vm() {
    static_assert(N >= 0 && N <= 63, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0x0 << 8));
  }
};

// Tile (slow, fast) of block `id` in a grid of at least nslow * nfast blocks;
// false for the blocks beyond.  Blocks are dealt to the 8 XCDs round robin:
// block id runs on XCD id mod 8, which takes one contiguous eighth of the
// tiles in an order that walks GROUP slow tiles by all fast ones, so that the
// 32 blocks resident on an XCD share their operands' tiles through its L2: a
// square of them reads the fewest (logits of 4096 tokens: 1.17 PFLOP/s with
// groups of 2, 1.30 with 4, 1.33 with 5; of 1777 tokens 4 are 3% ahead of 5;
// gradient of W best with 4, of the hidden states with 6, by 1 to 3%).
template <int GROUP>
__device__ __forceinline__ bool xcd_tile(int64_t id, int64_t nslow, int64_t nfast, int& slow,
                                         int& fast) {
  const int64_t total = nslow * nfast, per = (total + 7) / 8;
  const int64_t at = id / 8;
  const int64_t l = (id % 8) * per + at;
  if (at >= per || l >= total) return false;
  const int64_t g = l / (GROUP * nfast), w = l % (GROUP * nfast);
  const int64_t rows = nslow - GROUP * g < GROUP ? nslow - GROUP * g : GROUP;
  slow = static_cast<int>(GROUP * g + w % rows);
  fast = static_cast<int>(w / rows);
  return true;
}

}  // namespace fs
