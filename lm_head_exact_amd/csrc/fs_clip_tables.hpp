// fs_clip_tables.hpp -- gradient tensors as tables in kernel arguments: which
// block takes which elements (host side of fs_clip.hip; needs no device, so its
// tests run without one).
#pragma once

#include "fs_host.hpp"

namespace fs {

constexpr int kClipThreads = 256;
constexpr int kVec = 16;                // bytes a lane loads at once
constexpr int kUnroll = 4;
// Bytes of input per block: one round of loads, which streams best when written
// back (16 KB 596 us against 645 us with 64 KB); the norm's blocks take four
// times that of much input, to leave fewer sums.
constexpr int64_t kChunkBytes = kClipThreads * kVec * kUnroll;
constexpr int kTable = 96;              // 96 * 32 + ... bytes: below the 4 KB of kernel arguments
constexpr int32_t kMaxTensors = 65536;
constexpr int64_t kMaxLaunchBlocks = 0xFFFFFFFFll / kClipThreads;  // fewer than 2^32 threads

// Tensors, or stretches of one that does not fit a launch.
struct ClipTable {
  const void* in[kTable];
  void* out[kTable];
  int64_t numel[kTable];
  int32_t first[kTable + 1];  // first block of each tensor in this launch
  uint8_t dtype[kTable];
  int32_t n;
  int32_t base;               // chunk index of the launch's first block
  int32_t chunk;              // bytes per block
};

__host__ __device__ constexpr int type_bytes(int dtype) { return dtype == FS_FP32 ? 4 : 2; }

inline int64_t tensor_blocks(int64_t numel, int dtype, int64_t chunk) {
  const int64_t elems = chunk / type_bytes(dtype);
  return (numel + elems - 1) / elems;
}

// Fills tables for blocks of `chunk` bytes and calls launch(table, blocks) for
// each, in order.  A launch takes up to kTable tensors and kMaxLaunchBlocks
// blocks; a tensor that goes beyond is continued in the next one.
template <class F>
hipError_t for_each_table(const void* const* grads, void* const* out, const int64_t* numel,
                          const fs_dtype* dtypes, int32_t n, int64_t chunk, F launch) {
  ClipTable t;
  t.n = 0;
  t.base = 0;
  t.chunk = static_cast<int32_t>(chunk);
  int64_t blocks = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int64_t bytes = type_bytes(dtypes[i]), elems = chunk / bytes;
    for (int64_t at = 0; at < numel[i];) {
      const int64_t left = tensor_blocks(numel[i] - at, dtypes[i], chunk);
      const int64_t room = kMaxLaunchBlocks - blocks, take = left < room ? left : room;
      const char* in = static_cast<const char*>(grads[i]);
      char* to = static_cast<char*>(out ? out[i] : const_cast<void*>(grads[i]));
      t.in[t.n] = in + at * bytes;
      t.out[t.n] = to + at * bytes;
      t.numel[t.n] = take < left ? take * elems : numel[i] - at;
      t.dtype[t.n] = static_cast<uint8_t>(dtypes[i]);
      t.first[t.n] = static_cast<int32_t>(blocks);
      at += t.numel[t.n];
      blocks += take;
      t.first[++t.n] = static_cast<int32_t>(blocks);
      if (t.n == kTable || blocks == kMaxLaunchBlocks) {
        const hipError_t e = launch(t, static_cast<unsigned>(blocks));
        if (e != hipSuccess) return e;
        t.base += static_cast<int32_t>(blocks);
        t.n = 0;
        blocks = 0;
      }
    }
  }
  return t.n > 0 ? launch(t, static_cast<unsigned>(blocks)) : hipSuccess;
}

// Blocks of all tensors at the smaller chunk and fp32 (an upper bound), or -1.
// (Below 2^31 by more than the threads that step through their sums.)
inline int64_t max_chunks(const int64_t* numel, int32_t n) {
  if (n < 0 || n > kMaxTensors || (n > 0 && !numel)) return -1;
  int64_t c = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] > (int64_t{1} << 42)) return -1;
    c += tensor_blocks(numel[i], FS_FP32, kChunkBytes);
    if (c > 0x7FFFFFFF - 4096) return -1;
  }
  return c;
}

}  // namespace fs
