// Walks the slabs of rows up to the widest that an int counts as the row
// operators do, with the same index functions: every column is taken once, no
// column leaves 32 bits (UndefinedBehaviorSanitizer ends the program where one
// does), and lanes past the row see that they are.
#include <cstdio>
#include <initializer_list>

#include "moe_rows_index.hpp"

static int fails = 0;
#define CHECK(c, ...)                        \
  do {                                       \
    if (!(c) && fails++ < 20) {              \
      std::printf("line %d: %s: ", __LINE__, #c); \
      std::printf(__VA_ARGS__);              \
      std::printf("\n");                     \
    }                                        \
  } while (0)

// The columns of the slabs from `from` on: those inside the row.
static long long inside(int m, int slab, bool fours) {
  long long n = 0;
  for (int lane = 0; lane < 64; ++lane) {
    const moe::NormCols c = moe::slab_cols(fours, lane, slab);
    for (int at : {c.lo, c.hi}) {
      CHECK(at >= 0, "m %d slab %d lane %d", m, slab, lane);
      if (at < m) {
        CHECK(at + 3 < m, "m %d slab %d lane %d", m, slab, lane);
        n += 4;
      }
    }
  }
  return n;
}

int main() {
  constexpr int kMost = 0x7FFFFFFF - 7;  // the largest multiple of 8
  for (int m : {8, 504, 512, 520, 4088, 4096, 4104, 1 << 20, (1 << 20) + 8, 1 << 30, kMost - 4096, kMost - 4088, kMost - 1024,
                kMost - 512, kMost - 504, kMost - 496, kMost - 8, kMost})
    for (int fours = 0; fours < 2; ++fours) {
      const int slabs = moe::row_slabs(m);
      CHECK(512LL * slabs >= m && 512LL * (slabs - 1) < m, "m %d: %d slabs", m, slabs);
      // the combine's gradient: each wave's steps of two slabs, the first and the last ones
      int waves = (m / 8 + 127) / 128;
      if (waves > 4) waves = 4;
      const int skip = slabs > 64 ? (slabs - 32) / (2 * waves) * (2 * waves) : 0;  // slabs of whole steps left out
      long long n = 0;
      for (int wave = 0; wave < waves; ++wave)
        for (int slab = wave + skip; slab < slabs; slab += waves * 2)
          for (int v = 0; v < 2; ++v) n += inside(m, slab + v * waves, fours);
      CHECK(n == m - 512LL * skip, "m %d: %lld columns past slab %d", m, n, skip);
      // the combine: items of two slabs
      const int slices = (m / 8 + 127) / 128, first = slices > 16 ? slices - 16 : 0;
      n = 0;
      for (int s = first; s < slices; ++s)
        for (int v = 0; v < 2; ++v) n += inside(m, 2 * s + v, fours);
      CHECK(n == m - 1024LL * first, "m %d: %lld columns past slice %d", m, n, first);
    }
  if (fails) return 1;
  std::printf("wide rows ok\n");
  return 0;
}
