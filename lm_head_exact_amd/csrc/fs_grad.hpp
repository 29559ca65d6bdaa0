// fs_grad.hpp -- the gradient of the LM head that the training operators share
// (kernels in fs_logprob_grad.hip): rows that have a target are gathered, their
// dz is made in bf16 for a slice of the vocabulary at a time, and
//   dh = dz W,   dW = dz^T h
// read it back.  The targets' own terms are kept out of dz and added in fp32
// where the results are rounded.  Not installed; not part of the ABI.
#pragma once

#include <algorithm>
#include <cmath>

#include "fs_host.hpp"
#include "fs_internal.hpp"
#include "fs_score.hpp"

namespace fs {

// Per row that has a target, in order.
struct RowTerm {
  float inv_t;   // 1 / T
  float lse;     // of the scaled logits
  float coef;    // -g / T
  float target;  // g / T * (1 - p_target)
};

struct GradArgs {
  const __bf16 *h, *W;
  int32_t B, D, V, vocab_offset;
  const float *temperature, *logprob, *lse;
  const float* grad;  // null: the rows' terms are left to a later kernel
  const int32_t* ids;
  __bf16 *dh, *dW;    // either may be null
  // workspace
  int32_t* count;     // [2]: rows with a target; parts of the vocabulary for dh
  int32_t* slot;      // [B]: their place among them, or -1
  int32_t* row;       // [Bp]: the inverse
  int32_t* loc;       // [Bp]: target's row of W, or -1
  RowTerm* term;      // [Bp]
  __bf16* hz;         // [Bp][Dp]: their hidden states, zeros behind them
  __bf16* dz;         // [Bp][ldz]: of the slice
  float* slab;        // [max_splits][B][D] or null
  // targets by tile of 256 vocabulary rows
  int32_t* first;     // [V]: first place whose target the row is, or -1
  int32_t* list;      // [Bp]: places that have a target here, by tile
  int2* tile;         // [tiles]: begin and end in `list`
  float* side;        // [Bp][D]: dW rows of targets, at their first place
  float* wslab;       // [w_splits][V][D] where the rows are taken in parts for dW, or null
  int32_t Dp, Bp, ldz;
  int32_t v0, nv;     // the slice: rows v0 .. v0 + nv of W
  int32_t max_splits, hidden_tb, first_slice, w_splits;
};

constexpr int kGradPlaces = 32;  // places that dW takes at a time: dz is 0 behind the last one
constexpr int kTargetTile = 256;
constexpr int kTargetThreads = 1024;

// A row counts where it has a token; a token of another shard still gives
// every row of this one a gradient.
__device__ __forceinline__ bool has_token(int32_t id) { return id >= 0; }

__device__ __forceinline__ uint64_t pack_bf16(float x0, float x1, float x2, float x3) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  const bf16x4 v = {static_cast<__bf16>(x0), static_cast<__bf16>(x1), static_cast<__bf16>(x2),
                    static_cast<__bf16>(x3)};
  return __builtin_bit_cast(uint64_t, v);
}

constexpr int32_t kMaxGradB = 1 << 22;
constexpr int32_t kMaxGradD = 1 << 20;
// dz of one slice of the vocabulary.
constexpr int64_t kSliceBytes = int64_t{1} << 30;
constexpr int32_t kMaxSlice = 1 << 18;

inline int32_t target_tiles(int32_t V) {
  return static_cast<int32_t>((static_cast<int64_t>(V) + kTargetTile - 1) / kTargetTile);
}

// Parts of the rows for dW.  Its tiles of 256 vocabulary rows by 128 columns are few
// where both are small, and many rows leave each a long way: 6922 rows of 488 on 1633
// take 111 us in 28 blocks (a call 218 us, 139 in parts; 3990 of 256 on 1933 144 and 104,
// 8192 of 1024 on 4000 347 and 301).  A block's 32 rows take about half a microsecond;
// every part writes and reads V x D in fp32 at about 5 TB/s, and one launch more adds
// them up: taken where that saves a few microseconds.
inline int32_t weight_splits(int32_t B, int32_t D, int32_t V) {
  const int64_t tiles = (static_cast<int64_t>(V) + 255) / 256 * ((D + 127) / 128);
  if (tiles >= 256 || B < 512) return 1;
  const double whole = B / 64.0, each = 1.6e-6 * V * D;
  const int64_t s = std::min<int64_t>({static_cast<int64_t>(std::sqrt(whole / each)), 512 / tiles,
                                       B / 256});
  return s > 1 && whole - whole / s - each * s > 8.0 ? static_cast<int32_t>(s) : 1;
}

// Sizes and workspace of a call.  `whole`: dz is kept for the whole vocabulary, in
// slices of up to kMaxSlice rows one behind the other, instead of one slice of
// kSliceBytes at a time.  `parts`: dW may take the rows in parts.
struct GradPlan {
  int32_t Bp, Dp, slice, slices, splits, TB, w_splits;
  bool slabs;
  size_t count, slot, row, loc, term, hz, dz, slab, first, list, tile, side, wslab, total;
  GradPlan(int32_t B, int32_t D, int32_t V, bool whole_dz = false, bool parts = false) {
    TB = tile_tokens(B);
    Bp = static_cast<int32_t>(round_up(B, 256));
    Dp = static_cast<int32_t>(round_up(D, 64));
    int64_t s = whole_dz ? kMaxSlice : kSliceBytes / (2 * static_cast<int64_t>(Bp)) / 256 * 256;
    s = s < 256 ? 256 : s > kMaxSlice ? kMaxSlice : s;
    const int64_t whole = static_cast<int64_t>(round_up(V, 256));
    if (s >= whole) {
      s = whole;
    } else {  // equal slices
      const int64_t k = (whole + s - 1) / s;
      s = static_cast<int64_t>(round_up((whole + k - 1) / k, 256));
    }
    slice = static_cast<int32_t>(s);
    slices = static_cast<int32_t>((static_cast<int64_t>(V) + slice - 1) / slice);
    // at most as many parts for dh as make four rounds of its tiles, of at least
    // 256 vocabulary rows, with slabs of no more than 512 MiB
    const int64_t tiles = static_cast<int64_t>((B + TB - 1) / TB) * ((D + 255) / 256);
    const int64_t rows = slice < V ? slice : V;
    int64_t p = (1024 + tiles - 1) / tiles;
    p = std::min({p, rows / 256, (int64_t{512} << 20) / (4 * static_cast<int64_t>(B) * D)});
    splits = static_cast<int32_t>(p < 1 ? 1 : p);
    slabs = splits > 1 || slice < V;
    w_splits = parts && slices == 1 ? weight_splits(B, D, V) : 1;
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t o = at;
      at += round_up(bytes, 256);
      return o;
    };
    count = take(8);
    slot = take(4ull * B);
    row = take(4ull * Bp);
    loc = take(4ull * Bp);
    term = take(sizeof(RowTerm) * Bp);
    hz = take(2ull * Bp * Dp);
    dz = take(2ull * Bp * slice * (whole_dz ? slices : 1));
    slab = take(slabs ? 4ull * splits * B * D : 0);
    first = take(4ull * V);
    list = take(4ull * Bp);
    tile = take(sizeof(int2) * target_tiles(V));
    side = take(w_splits > 1 ? 0 : 4ull * Bp * D);
    wslab = take(w_splits > 1 ? 4ull * w_splits * V * D : 0);
    total = at;
  }
};

inline bool grad_sizes_ok(int32_t B, int32_t D, int32_t V) {
  return B >= 0 && D >= 8 && D % 8 == 0 && V >= 1 && B <= kMaxGradB && D <= kMaxGradD &&
         V <= kMaxVocab;
}
// Whether every launch's grid holds fewer than 2^32 threads.
bool grad_grids_fit(int32_t B, int32_t D, int32_t V, const GradPlan& p, bool dh, bool dW);

// Sets the workspace's arrays and the sizes that follow from the plan.
void grad_workspace(GradArgs& a, const GradPlan& p, char* ws);

// Rows with a target, their places and the parts that dh is taken in; copies of their
// hidden states and, with a gradient, their terms; dh of the others is 0; for dW the
// targets by tile of the vocabulary.
hipError_t launch_grad_rows(const GradArgs& a, hipStream_t stream);
// dW and dh of the slice v0, nv from its dz.
hipError_t launch_grad_products(const GradArgs& a, hipStream_t stream);
// The targets' terms and the parts of dh, once every slice is through.
hipError_t launch_grad_finish(const GradArgs& a, hipStream_t stream);

}  // namespace fs
