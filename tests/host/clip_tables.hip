// Walks the tables that for_each_table makes, on the host, and checks that the
// launches stay below 2^32 threads and their blocks cover every tensor once, in
// order.  Nothing is launched: the pointers are numbers.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "fs_clip_tables.hpp"

using namespace fs;

#define CHECK(c)                              \
  do {                                        \
    if (!(c)) {                               \
      printf("%s: line %d: %s\n", name, __LINE__, #c); \
      exit(1);                                \
    }                                         \
  } while (0)

static void tables(const char* name, const std::vector<int64_t>& numel, const std::vector<int>& types,
                   int64_t chunk, bool in_place) {
  const int n = static_cast<int>(numel.size());
  std::vector<const void*> in(n);
  std::vector<void*> out(n);
  std::vector<fs_dtype> dt(n);
  for (int i = 0; i < n; ++i) {
    in[i] = reinterpret_cast<const void*>((int64_t{i} + 1) << 46);
    out[i] = reinterpret_cast<void*>(((int64_t{i} + 1) << 46) + (int64_t{1} << 45));
    dt[i] = static_cast<fs_dtype>(types[i % types.size()]);
  }
  int64_t base = 0, launches = 0;
  int i = 0;        // tensor and element that come next
  int64_t at = 0;
  auto skip_empty = [&] { while (i < n && numel[i] == 0) ++i; };
  skip_empty();
  const hipError_t e = for_each_table(in.data(), in_place ? nullptr : out.data(), numel.data(),
                                      dt.data(), n, chunk, [&](const ClipTable& t, unsigned blocks) {
    ++launches;
    CHECK(t.n >= 1 && t.n <= kTable && blocks >= 1);
    CHECK(static_cast<unsigned long long>(blocks) * kClipThreads < (1ull << 32));
    CHECK(t.base == base && t.chunk == chunk && t.first[0] == 0 &&
          t.first[t.n] == static_cast<int64_t>(blocks));
    for (int k = 0; k < t.n; ++k) {
      const int bytes = type_bytes(dt[i]);
      const int64_t elems = chunk / bytes, have = t.first[k + 1] - t.first[k];
      CHECK(t.dtype[k] == dt[i] && t.numel[k] >= 1);
      CHECK(t.in[k] == static_cast<const char*>(in[i]) + at * bytes);
      CHECK(t.out[k] == static_cast<const char*>(in_place ? in[i] : out[i]) + at * bytes);
      CHECK(have * elems >= t.numel[k] && (have - 1) * elems < t.numel[k]);
      at += t.numel[k];
      CHECK(at <= numel[i]);
      if (at < numel[i]) {
        CHECK(t.numel[k] % elems == 0);  // continued at a whole chunk
      } else {
        at = 0;
        ++i;
        skip_empty();
      }
    }
    base += blocks;
    return hipSuccess;
  });
  CHECK(e == hipSuccess && i == n && at == 0);
  CHECK(base <= max_chunks(numel.data(), n) * (kChunkBytes > chunk ? 2 : 1));
  printf("%s: %lld launches, %lld blocks\n", name, static_cast<long long>(launches),
         static_cast<long long>(base));
}

int main() {
  const int64_t G = int64_t{1} << 30;
  for (int64_t chunk : {kChunkBytes, 4 * kChunkBytes})
    for (bool in_place : {true, false}) {
      tables("nothing", {}, {0}, chunk, in_place);
      tables("empty", {0, 0}, {0}, chunk, in_place);
      tables("small", {1, 0, 4096, 4097, 32768, 0}, {0, 1, 2}, chunk, in_place);
      tables("95", std::vector<int64_t>(95, 13), {2}, chunk, in_place);
      tables("96", std::vector<int64_t>(96, 13), {2}, chunk, in_place);
      tables("97, the last empty", [] { std::vector<int64_t> v(97, 13); v[96] = 0; return v; }(), {1},
             chunk, in_place);
      tables("300", std::vector<int64_t>(300, 70001), {0, 2}, chunk, in_place);
      tables("64 G elements, fp32", {64 * G}, {2}, chunk, in_place);
      tables("64 G elements less some", {64 * G - 4096, 5, 64 * G - 4097}, {2, 0}, chunk, in_place);
      tables("a launch exactly", {kMaxLaunchBlocks * (kChunkBytes / 4), 1}, {2}, chunk, in_place);
      tables("several launches", {300 * G + 77, 3, 200 * G + 1, 0, 9}, {0, 2, 1}, chunk, in_place);
      tables("many large ones", std::vector<int64_t>(90, 3 * G + 1), {0, 2}, chunk, in_place);
    }
  printf("every block in place\n");
  return 0;
}
