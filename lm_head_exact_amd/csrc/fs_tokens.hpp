// fs_tokens.hpp -- how a team of threads walks the tokens of a sequence
// (host and device: the walk is also compiled for the host and tested there).
#pragma once

#include <hip/hip_runtime.h>

namespace fs {

// Token loads in flight per thread.
constexpr int kAhead = 4;

// Calls f(t) for the tokens [t0 + lane, t1) strided by `team`, with kAhead of
// them loaded by load(t) at a time; 0 <= t0, t1.  The counter is unsigned: the
// step behind the last token, at most team * kAhead past it, may lie beyond
// 2^31 - 1 and stays below 2^32.
template <class Load, class F>
__host__ __device__ __forceinline__ void each_token(int t0, int t1, int lane, int team, Load load,
                                                    F f) {
  const unsigned end = t1, step = team;
  for (unsigned t = static_cast<unsigned>(t0) + lane; t < end; t += step * kAhead) {
    decltype(load(0)) v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (t + u * step < end) v[u] = load(static_cast<int>(t + u * step));
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (t + u * step < end) f(static_cast<int>(t + u * step), v[u]);
  }
}

}  // namespace fs
