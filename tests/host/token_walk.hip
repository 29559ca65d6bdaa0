// Walks token ranges with each_token on the host and checks that the lanes of
// a team visit every token once, loaded before it is handed on, and nothing else.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "fs_tokens.hpp"

static void walk(int t0, int t1, int team) {
  std::vector<int> seen(t1 - t0, 0);
  for (int lane = 0; lane < team; ++lane)
    fs::each_token(t0, t1, lane, team, [](int t) { return t; },
                   [&](int t, int loaded) {
                     if (t < t0 || t >= t1 || loaded != t || seen[t - t0]++ != 0) {
                       printf("[%d, %d) by %d: lane %d visits %d\n", t0, t1, team, lane, t);
                       exit(1);
                     }
                   });
  for (int i = 0; i < t1 - t0; ++i)
    if (seen[i] != 1) {
      printf("[%d, %d) by %d: token %d left out\n", t0, t1, team, t0 + i);
      exit(1);
    }
}

int main() {
  const int lengths[] = {0, 1, 63, 64, 255, 256, 257, 1023, 1024, 1025, 5000};
  for (int team : {64, 256})
    for (int n : lengths) {
      walk(0, n, team);
      walk(12345, 12345 + n, team);
      // up to the last token that 32 bits count, and up to a little below it
      for (int below : {0, 1, 200, 255, 256, 1000, 1023, 1024, 1025})
        walk(INT32_MAX - below - n, INT32_MAX - below, team);
    }
  printf("every token once\n");
  return 0;
}
