// fs_score.hpp -- shared parts of the token log-probability operators: the
// epilogue that turns a block's logits into one log-sum-exp partial per
// token, and the arguments of its kernels.
//
// Scaled logits t_v = z_v * fp32(1/T) (rows whose T is not positive: t = z).
// A token's partial over a block of vocabulary rows is the pair (m, s) with
// sum exp(t_v) = s exp(m) over the rows that are not its target; the target's
// own t goes to a separate array.  With L the log-sum-exp of the others,
//   log p(target) = -log(1 + exp(L - t_target)),
// which keeps its relative accuracy where the target is nearly certain;
// t_target - logsumexp(all) would cancel there.
#pragma once

#include <atomic>

#include "fs_tile.hpp"

namespace fs {

// Most rows of W in a call: row numbers a tile past the last stay below 2^31.
constexpr int32_t kMaxVocab = 0x7FFFFFFF - 512;

struct ScoreArgs {
  Operand w, h;             // W [V][D] (or fragment order), h [B][D]
  int32_t B, D, V, vocab_offset, shift;  // shift: rows before row 0 in the grid (fragment order)
  const float* temperature;  // [B] or null (all 1)
  const int32_t* ids;        // [B]
  float2* part;              // [S][B]
  float* target;             // [B]: the target's scaled logit
  int32_t S;
};

__device__ __forceinline__ float score_inv_t(const float* temperature, int b) {
  return temperature != nullptr ? row_inv_temperature(temperature[b]) : 1.0f;
}

// The target's local vocabulary row, or -1 (no target, or another shard's).
__device__ __forceinline__ int target_row(int32_t id, int32_t vocab_offset, int32_t V) {
  if (id < vocab_offset) return -1;  // (vocab_offset >= 0, so negative ids too)
  const int loc = id - vocab_offset;
  return loc < V ? loc : -1;
}

// (m, s) of the union of two disjoint sets of rows.  m is -FLT_MAX where s is 0.
__device__ __forceinline__ void pair_merge(float& m, float& s, float om, float os) {
  const float nm = fmaxf(m, om);
  s = s * LseAcc::ex(m - nm) + os * LseAcc::ex(om - nm);
  m = nm;
}
__device__ __forceinline__ void pair_xor(float& m, float& s, int mask) {
  const float om = __shfl_xor(m, mask, kWave), os = __shfl_xor(s, mask, kWave);
  pair_merge(m, s, om, os);
}

// Folds the wave's logits of one token into (m, s): z[i][r] is vocabulary row
// row0 + 16 i + r + 4 kb.  All values are in registers, so the maximum comes
// first and each logit costs one multiply-add and one exp2.  `plain` (the
// same on all lanes): no row of the wave is outside [0, V) or any of its
// tokens' target, so nothing is excluded.
template <int MR, class Z>
__device__ __forceinline__ void fold_logits(const Z& z, int row0, int32_t V, int loc, bool plain,
                                            float inv_t, float& m, float& s, float& zt,
                                            bool& has_zt) {
  const int kb = (threadIdx.x & (kWave - 1)) >> 4;
  const float c = inv_t * 1.44269504088896341f;  // log2(e) / T
  float mz = LseAcc::kMasked, sum = 0.0f;
  if (plain) {
    static_for<MR>([&](auto i) FS_INLINE {
      const f32x4 x = z(i);
      mz = fmaxf(fmaxf(mz, fmaxf(x[0], x[1])), fmaxf(x[2], x[3]));
    });
    const float off = mz * c;
    static_for<MR>([&](auto i) FS_INLINE {
      const f32x4 x = z(i);
      static_for<4>([&](auto r) FS_INLINE {
        sum += __builtin_amdgcn_exp2f(__builtin_fmaf(x[decltype(r)::value], c, -off));
      });
    });
  } else {
    auto keep = [&](int v) FS_INLINE {
      return static_cast<uint32_t>(v) < static_cast<uint32_t>(V) && v != loc;
    };
    static_for<MR>([&](auto i) FS_INLINE {
      const f32x4 x = z(i);
      static_for<4>([&](auto r) FS_INLINE {
        const int v = row0 + 16 * static_cast<int>(i) + 4 * kb + static_cast<int>(r);
        if (v == loc && loc >= 0) {
          zt = x[decltype(r)::value] * inv_t;
          has_zt = true;
        }
        mz = keep(v) ? fmaxf(mz, x[decltype(r)::value]) : mz;
      });
    });
    const float off = mz * c;
    static_for<MR>([&](auto i) FS_INLINE {
      const f32x4 x = z(i);
      static_for<4>([&](auto r) FS_INLINE {
        const int v = row0 + 16 * static_cast<int>(i) + 4 * kb + static_cast<int>(r);
        // the exponential of an excluded row may be anything: not added
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[decltype(r)::value], c, -off));
        sum += keep(v) ? e : 0.0f;
      });
    });
  }
  pair_merge(m, s, mz == LseAcc::kMasked ? mz : mz * inv_t, sum);
}

// ---- tiles of the logits (W is operand A, h operand B) ----
// L: the layout of W.  Tall: 256 vocabulary rows by 64, 128 or 256 tokens.
// Short, 4 waves, two blocks per CU: 64 by 64, 64 by 128, 128 by 128.
template <int L, int TB> struct TallTile;
template <int L> struct TallTile<L, 64> { using T = Tile<L, kKC, 8, 1, 2, 4, 4, 64, L == kFrag>; };
template <int L> struct TallTile<L, 128> { using T = Tile<L, kKC, 4, 2, 4, 4, 3, 64, L == kFrag>; };
template <int L> struct TallTile<L, 256> { using T = Tile<L, kKC, 2, 4, 8, 4, 2>; };
template <int L, int TB> struct ShortTile;
template <int L> struct ShortTile<L, 64> { using T = Tile<L, kKC, 4, 1, 1, 4, 4, 64, L == kFrag>; };
template <int L> struct ShortTile<L, 128> { using T = Tile<L, kKC, 4, 1, 1, 8, 3, 64, L == kFrag>; };
template <int L> struct ShortTile<L, 256> { using T = Tile<L, kKC, 2, 2, 4, 4, 2>; };
constexpr int kTallRows = 256, kMinTileRows = 64;  // vocabulary rows of the tall tiles, and of any

enum class LogitsTile { kTall64, kTall128, kTall256, kShort64, kShort128, kShort256 };

inline int tile_tokens(int32_t B) { return B <= 64 ? 64 : B <= 128 ? 128 : 256; }

// The tile for B tokens and V rows: the largest whose grid keeps three quarters
// of the CUs busy.  Large tiles move less per product (512 tokens on 128256
// rows of 4096: 475 us tall, 608 short); a grid of few leaves CUs idle (the
// same tokens on 16032 rows of 8192: 195 us tall, 144 short), and where even
// the short ones are few their k loops alone take the time (1024 tokens on
// 1000 rows of 8192: 84 us by 128 x 128, 28 by 64 x 64).
inline LogitsTile logits_tile(int32_t B, int32_t V) {
  constexpr int64_t kBlocks = 192;
  auto grid = [&](int rows, int tokens) {
    return (static_cast<int64_t>(V) + rows - 1) / rows * ((B + tokens - 1) / tokens);
  };
  const int TB = tile_tokens(B);
  if (grid(kTallRows, TB) >= kBlocks)
    return TB == 64    ? LogitsTile::kTall64
           : TB == 128 ? LogitsTile::kTall128
                       : LogitsTile::kTall256;
  if (TB == 256 && grid(128, 128) >= kBlocks) return LogitsTile::kShort256;
  if (TB == 128 && grid(64, 128) >= kBlocks) return LogitsTile::kShort128;
  return LogitsTile::kShort64;
}

inline bool is_tall(LogitsTile t) { return t <= LogitsTile::kTall256; }

// Raises a kernel's dynamic-LDS limit, once per device (the limit is a device's
// own).  Each kernel keeps its own record.
struct SmemRaised {
  static constexpr int kMaxDevices = 64;
  std::atomic<bool> on[kMaxDevices];
};
template <class Kernel>
hipError_t raise_smem(Kernel kernel, size_t smem, SmemRaised& raised) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const bool known = dev >= 0 && dev < SmemRaised::kMaxDevices;
  if (known && raised.on[dev].load(std::memory_order_acquire)) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == hipSuccess && known) raised.on[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace fs
