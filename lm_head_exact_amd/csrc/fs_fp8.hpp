// fs_fp8.hpp -- the LM head in 8-bit floating point: shared parts of the
// quantising kernels, the streaming kernels (few rows) and the block-tiled ones.
//
// Format.  Values are e4m3 (no infinities, largest 448, NaN 0x7F), rounded to
// nearest even.  A block of 128 columns (weights: of 128 rows too) shares the
// scale 2^e, stored as one byte e + 127 (e8m0), with the least e >= -110 for
// which no finite entry exceeds 448 * 2^e; e = 0 for a block of zeros.  Entries
// that are not finite become NaN.  A power of two costs no precision (the values
// are floating point: the scale moves exponents only, and up to one binade of
// the smallest ones), makes quantising exact but for its one rounding, and is
// what the matrix cores take (v_mfma_scale_f32_32x32x64_f8f6f4): no multiply by
// scales follows the products.
//
// W lies in fragment order: groups of 16 rows, 64 columns at a time as the 64
// lanes' 16 bytes: byte ((g * D/64 + s) * 64 + l) * 16 + j holds
// W[16 g + l mod 16][64 s + 16 (l / 16) + j], rows past V zero.
#pragma once

#include "fs_score.hpp"

namespace fs {

constexpr int kQuantBlock = 128;
constexpr int32_t kMaxFp8D = 1 << 14;
constexpr int32_t kMaxFp8B = 1 << 22;

inline int32_t fp8_groups(int32_t V) {
  return static_cast<int32_t>((static_cast<int64_t>(V) + 15) / 16);
}
__host__ __device__ inline int32_t quant_blocks(int32_t n) {
  return (n - 1) / kQuantBlock + 1;
}

// e + 127 of a block whose largest finite magnitude has these bf16 bits.
__device__ __forceinline__ int scale_byte(uint32_t amax) {
  // 2^(x - 127) <= amax < 2^(x - 126), x its exponent field; 448 = 1.75 * 2^8
  const int e = static_cast<int>(amax >> 7) - 8 + ((amax & 0x7F) > 0x60);
  return amax == 0 ? 127 : max(e, 127 - 110);
}
// 2^e and 2^-e of a scale byte (17 to 247).
__device__ __forceinline__ float scale_up(int byte) { return __int_as_float(byte << 23); }
__device__ __forceinline__ float scale_down(int byte) { return __int_as_float((254 - byte) << 23); }

// The larger of two magnitudes as bf16 bits, what is not finite left out.
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t bits) {
  const uint32_t a = bits & 0x7FFF;
  return a < 0x7F80 ? max(m, a) : m;
}
__device__ __forceinline__ uint32_t finite_max2(uint32_t m, uint32_t pair) {
  return finite_max(finite_max(m, pair), pair >> 16);
}
// Both halves' magnitudes, whatever they are: two instructions per pair.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 any_max2(u16x2 m, uint32_t pair) {
  return __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, pair & 0x7FFF7FFFu));
}

// Two pairs of bf16 to four e4m3 bytes, each times `down`.  (Finite entries end
// up at 448 at most; infinities and NaN convert to NaN.)
__device__ __forceinline__ uint32_t to_e4m3(uint32_t p0, uint32_t p1, float down) {
  const float x0 = __uint_as_float(p0 << 16) * down, x1 = __uint_as_float(p0 & 0xFFFF0000u) * down;
  const float x2 = __uint_as_float(p1 << 16) * down, x3 = __uint_as_float(p1 & 0xFFFF0000u) * down;
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(x0, x1, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(x2, x3, v, true);
  return static_cast<uint32_t>(v);
}

// Eight e4m3 bytes times 2^e as bf16: exact (four significant bits).
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi, float up) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, up, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, up, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, up, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, up, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// What a kernel makes of the logits.
enum Fp8Out { kLogitsBf16, kLogitsF32, kTokenScores, kSamples };

struct Fp8Args {
  const uint8_t* w;       // fragment order
  const uint8_t* wscale;  // [quant_blocks(V)][KB]
  const __bf16* h;        // [B][D]
  int32_t B, D, V, KB, vocab_offset;
  // h in 8 bits (tiles): [B][Dp], zeros past D; scales [KB][Bp]
  uint8_t* hq;
  uint8_t* hscale;
  int32_t Dp, Bp;
  const float* temperature;
  // token scores: as fs_token_logprobs
  const int32_t* ids;
  float2* part;   // [S][B]
  float* target;  // [B]
  // samples: as fs_sample
  uint64_t seed, step;
  float* part_val;    // [B][S]
  int32_t* part_idx;  // [B][S]
  // logits [B][V], rows ld elements apart; lines: every row starts a line of 128 bytes
  void* out;
  int64_t ld;
  bool lines;
  int32_t S;
};

// Whether the streaming kernels take the call; their most blocks.
inline bool fp8_streams(int32_t B, int32_t D) {
  return (B <= 16 && D <= 8192) || (B <= 32 && D <= 5120);
}
constexpr int kMaxFp8StreamBlocks = 2048;

// Tiles: the bf16 products' shapes but 64 x 128, with their ring's slots of 128 k.
struct Fp8TileShape {
  LogitsTile tile;
  int32_t rows, tokens, slots;
};
constexpr Fp8TileShape kFp8TileShapes[] = {
    {LogitsTile::kTall64, 256, 64, 3},    {LogitsTile::kTall128, 256, 128, 3},
    {LogitsTile::kTall256, 256, 256, 2},  {LogitsTile::kShort64, 64, 64, 3},
    {LogitsTile::kShort256, 128, 128, 2}};
constexpr size_t kFp8Lds = 160 * 1024;

// LDS of a tile: the ring, and the scales of its tokens and of its blocks of rows.
inline size_t fp8_lds(const Fp8TileShape& c, int32_t D) {
  return static_cast<size_t>(c.slots) * (c.rows + c.tokens) * kQuantBlock +
         static_cast<size_t>(quant_blocks(D)) * (c.tokens + (c.rows + 127) / 128);
}

// Microseconds of a grid of c's blocks on 16032 rows of 8192, by rounds of 256 blocks
// (one block of the tall tiles per CU; of 128 x 128 two, of 64 x 64 three).  Measured
// there: 256 x 64 39 and 70 (one round, two), 256 x 128 46 to 56 and 101 to 121, 256 x
// 256 78 to 103 and 188 to 201, 64 x 64 25, 31, 54, 76 and 110 (rounds 1, 2, 4, 6, 9),
// 128 x 128 55, 55, 103 and 122 (1 to 4).  Over 72 calls (40 to 2048 tokens on 2001 to
// 151936 rows of 1024 to 8192) the tile that it takes is 1.2% behind the best one on
// average, by the bf16 products' costs 6%; at most 15%, where memory bounds the call (100
// tokens on 32064 rows of 4096: 31 us by 256 x 64, 27 by 256 x 128).
inline int64_t fp8_tile_cost(const Fp8TileShape& c, int64_t B, int64_t V) {
  const int64_t blocks = (V + c.rows - 1) / c.rows * ((B + c.tokens - 1) / c.tokens);
  const int64_t rounds = (blocks + 255) / 256;
  switch (c.tile) {
    case LogitsTile::kTall64: return 38 * rounds;
    case LogitsTile::kTall128: return 57 * rounds;
    case LogitsTile::kTall256: return 100 * rounds;
    case LogitsTile::kShort64: return rounds == 1 ? 25 : 5 + 12 * rounds;
    default: return 60 * ((rounds + 1) / 2);
  }
}

// The tile for a call: the cheapest whose scales fit in LDS beside its ring (64 x 64
// always does).
inline LogitsTile fp8_tile(int32_t B, int32_t D, int32_t V) {
  LogitsTile best = LogitsTile::kShort64;
  int64_t least = INT64_MAX;
  for (const Fp8TileShape& c : kFp8TileShapes) {
    if (fp8_lds(c, D) > kFp8Lds) continue;
    const int64_t cost = fp8_tile_cost(c, B, V);
    if (cost < least) {
      least = cost;
      best = c.tile;
    }
  }
  return best;
}

hipError_t launch_quantize_weights(const __bf16* W, int32_t V, int32_t D, bool packed, uint8_t* q,
                                   uint8_t* scale, hipStream_t stream);
hipError_t launch_pack_fp8(const uint8_t* q, int32_t V, int32_t D, uint8_t* packed,
                           hipStream_t stream);
// h in 8 bits; with ids also every token's scaled logit.
hipError_t launch_quantize_rows(const Fp8Args& a, hipStream_t stream);
// Every one sets a.S.
hipError_t stream_logits_bf16(Fp8Args& a, hipStream_t stream);
hipError_t stream_logits_f32(Fp8Args& a, hipStream_t stream);
hipError_t stream_scores(Fp8Args& a, hipStream_t stream);
hipError_t stream_samples(Fp8Args& a, hipStream_t stream);
hipError_t tile_logits_bf16(Fp8Args& a, hipStream_t stream);
hipError_t tile_logits_f32(Fp8Args& a, hipStream_t stream);
hipError_t tile_scores(Fp8Args& a, hipStream_t stream);
hipError_t tile_samples(Fp8Args& a, hipStream_t stream);

}  // namespace fs
