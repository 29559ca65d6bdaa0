// Reads lines "B V some" and prints the logits' tile that the library's rule
// takes for them: its vocabulary rows and tokens.
#include <cstdio>

#include "fs_score.hpp"

int main() {
  int B, V, some;
  while (scanf("%d %d %d", &B, &V, &some) == 3) {
    const fs::LogitsTile t = fs::logits_tile(B, V, some != 0);
    printf("%d %d\n", fs::rows_of(t), fs::tokens_of(t));
  }
  return 0;
}
