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
//
// Logits of -inf add nothing (exp gives 0); NaN or +inf among them gives NaN.
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

// What is taken from the exponents of a lane's logits, whose maximum is mz: 0
// where that is -inf (the maximum starts at kMasked), for which the product
// would make -inf - (-inf) of them.
__device__ __forceinline__ float exponent_offset(float mz, float c) {
  return mz == LseAcc::kMasked ? 0.0f : mz * c;
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
    const float off = exponent_offset(mz, c);
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
    const float off = exponent_offset(mz, c);
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
// Short, 4 waves, two blocks per CU: 64 by 64, 64 by 128, 128 by 128.  NTA: W's
// loads are non-temporal.
template <int L, int TB, bool NTA = false> struct TallTile;
template <int L, bool NTA> struct TallTile<L, 64, NTA> { using T = Tile<L, kKC, 8, 1, 2, 4, 4, 64, NTA>; };
template <int L, bool NTA> struct TallTile<L, 128, NTA> { using T = Tile<L, kKC, 4, 2, 4, 4, 3, 64, NTA>; };
template <int L, bool NTA> struct TallTile<L, 256, NTA> { using T = Tile<L, kKC, 2, 4, 8, 4, 2, 64, NTA>; };
template <int L, int TB, bool NTA = false> struct ShortTile;
template <int L, bool NTA> struct ShortTile<L, 64, NTA> { using T = Tile<L, kKC, 4, 1, 1, 4, 4, 64, NTA>; };
template <int L, bool NTA> struct ShortTile<L, 128, NTA> { using T = Tile<L, kKC, 4, 1, 1, 8, 3, 64, NTA>; };
template <int L, bool NTA> struct ShortTile<L, 256, NTA> { using T = Tile<L, kKC, 2, 2, 4, 4, 2, 64, NTA>; };
constexpr int kTallRows = 256, kMinTileRows = 64;  // vocabulary rows of the tall tiles, and of any

enum class LogitsTile { kTall64, kTall128, kTall256, kShort64, kShort128, kShort256 };

inline int tile_tokens(int32_t B) { return B <= 64 ? 64 : B <= 128 ? 128 : 256; }

// The tile for B tokens and V rows: the one whose grid takes the least time.  A
// tall tile's block has a CU to itself, so its grid takes whole rounds of 256
// blocks; of the short ones, two share a CU, and their grids take about a round
// and a half of its cost for two.  The costs are in hundredths of a round of
// 256 x 64 tiles, from 16032 rows of 8192: a round of 256 x 64, 256 x 128 and
// 256 x 256 takes 91, 115 and 209 us (252 blocks each), 251, 502 and 1004
// blocks of 64 x 64 take 49, 68 and 123 us, of 64 x 128 60, 104 and 184, and
// 252, 504 and 1008 of 128 x 128 119, 138 and 252.  256 x 128 is given a little
// more: of two alike, 256 x 256 reads less.  (256 tokens there: 91 us by
// 256 x 64, 117 by 128 x 128; 768 tokens: 194 us by 256 x 256, 222 by 128 x 128;
// 1024 tokens on 1000 rows: 90 us by 128 x 128, 37 by 64 x 64.)  The costs do not
// see D: where it is small a block's prologue and epilogue weigh more than there.
struct TileShape {
  LogitsTile tile;
  int32_t rows, tokens;
};
constexpr TileShape kTileShapes[] = {
    {LogitsTile::kTall64, 256, 64},   {LogitsTile::kTall128, 256, 128},
    {LogitsTile::kTall256, 256, 256}, {LogitsTile::kShort64, 64, 64},
    {LogitsTile::kShort128, 64, 128}, {LogitsTile::kShort256, 128, 128}};

inline int64_t tile_cost(const TileShape& c, int64_t B, int64_t V) {
  const int64_t blocks = (V + c.rows - 1) / c.rows * ((B + c.tokens - 1) / c.tokens);
  const int64_t rounds = (blocks + 255) / 256;
  switch (c.tile) {
    case LogitsTile::kTall64: return 100 * rounds;
    case LogitsTile::kTall128: return 132 * rounds;
    case LogitsTile::kTall256: return 230 * rounds;
    case LogitsTile::kShort64: return 22 + 30 * rounds;
    case LogitsTile::kShort128: return 25 + 48 * rounds;
    default: return 148 * (rounds / 2) + 125 * (rounds % 2);
  }
}

// `some`: any share of the B tokens may be without a target and left out, which
// the device alone knows: the least cost of half, three quarters and, twice, all
// of them together (513 tokens on 16032 rows of 8192, of which 385 count: 107 us by 256
// x 128, 190 by 256 x 256, which would be the best for all of them).
inline LogitsTile logits_tile(int32_t B, int32_t V, bool some = false) {
  LogitsTile best = LogitsTile::kTall64;
  int64_t least = INT64_MAX;
  for (const TileShape& c : kTileShapes) {
    const int64_t b = B;
    int64_t cost = tile_cost(c, b, V);
    if (some) cost = 2 * cost + tile_cost(c, (b + 1) / 2, V) + tile_cost(c, (3 * b + 3) / 4, V);
    if (cost < least) {
      least = cost;
      best = c.tile;
    }
  }
  return best;
}

inline int tokens_of(LogitsTile t) {
  return t == LogitsTile::kTall64 || t == LogitsTile::kShort64 ? 64
         : t == LogitsTile::kTall256                           ? 256
                                                               : 128;
}

inline bool is_tall(LogitsTile t) { return t <= LogitsTile::kTall256; }

inline int threads_of(LogitsTile t) { return is_tall(t) ? 512 : 256; }
inline int rows_of(LogitsTile t) { return kTileShapes[static_cast<int>(t)].rows; }

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
