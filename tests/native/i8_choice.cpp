// Reads lines "rows K N experts cus" and prints the kernel that the int8
// product takes for each, and whether its weights are read as not to be kept
// (with w on a line's border).
#include <cstdio>

#include "moe_rows_index.hpp"

int main() {
  static const char* const names[] = {"32x256x3",  "64x256x3",  "32x256x2", "64x256x2", "256x256x2", "128x256x3",
                                      "128x128x4", "64x128x3", "64x64x4",  "ring16",   "ring64",    "ring32"};
  static_assert(sizeof names / sizeof *names == moe::kI8Kernels, "a name for every kernel");
  int R, K, N, E, cus;
  while (std::scanf("%d %d %d %d %d", &R, &K, &N, &E, &cus) == 5) {
    const moe::I8Choice c = moe::choose_i8(R, N, E, cus);
    std::printf("%s %d %d\n", names[c.kernel], c.once, c.once && moe::i8_weights_once(nullptr, K, N, E));
  }
  return 0;
}
