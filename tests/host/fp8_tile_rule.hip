// Reads lines "B D V" and prints the 8-bit head's tile that the library's rule takes
// for them (its vocabulary rows and tokens) and that tile's LDS.
#include <cstdio>

#include "fs_fp8.hpp"

int main() {
  int B, D, V;
  while (scanf("%d %d %d", &B, &D, &V) == 3) {
    const fs::LogitsTile t = fs::fp8_tile(B, D, V);
    for (const fs::Fp8TileShape& c : fs::kFp8TileShapes)
      if (c.tile == t) printf("%d %d %zu\n", c.rows, c.tokens, fs::fp8_lds(c, D));
  }
  return 0;
}
