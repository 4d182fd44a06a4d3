// Checks on the host that the fp32 reads of the gated feed-forward block's products meet no LDS
// bank twice in a cycle (64 banks of 4 bytes): ds_read_b32 of lines by reduction step takes 32 lanes
// a cycle, ds_read_b128 of rows 16 lanes.
#include <cstdio>
#include <set>

#include "moe_gated_index.hpp"

static int fails = 0;

template <class At>
static void distinct(const char* what, int lanes, int bytes, At at) {
  for (int first = 0; first < 64; first += lanes) {
    std::set<int> banks;
    for (int l = first; l < first + lanes; ++l)
      for (int b = 0; b < bytes; b += 4) banks.insert((at(l) + b) / 4 % 64);
    if ((int)banks.size() != lanes * bytes / 4 && fails++ < 20)
      std::printf("%s, lanes from %d: %zu of %d banks\n", what, first, banks.size(), lanes * bytes / 4);
  }
}

int main() {
  for (int ks = 0; ks < 4; ++ks) {
    for (int i = 0; i < 4; ++i) distinct("by step", 32, 4, [&](int l) { return moe::step_read_f32(l, ks, i); });
    distinct("by row", 16, 16, [&](int l) { return moe::operand32(l, ks); });
  }
  if (fails) return 1;
  std::printf("gated banks check ok\n");
  return 0;
}
