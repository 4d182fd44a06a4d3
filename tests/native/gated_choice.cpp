// Reads lines "bf16 rows m p E cus" and prints, for every product of the gated feed-forward
// block, the kernel that it takes: the tile (rows x weight lines x stages of its ring), the
// number of shares of its reduction, whether the weights are read as not to be kept, whether
// the hidden rows come in two parts, and the stages of its reduction (of the weight gradients:
// of an expert's mean rows).
#include <cstdio>

#include "moe_gated_index.hpp"

int main() {
  static const char* const names[] = {"256x256x2", "128x256x3", "128x128x2", "64x128x3", "32x256x2", "32x256x3", "32x128x2"};
  static_assert(sizeof names / sizeof *names == moe::kGatedTiles, "a name for every tile");
  int bf16, R, m, p, E, cus;
  while (std::scanf("%d %d %d %d %d %d", &bf16, &R, &m, &p, &E, &cus) == 6) {
    const int steps = moe::stage_steps(bf16 ? 2 : 4);
    const int sm = (m + steps - 1) / steps, sp = (p + steps - 1) / steps;
    const bool pair = moe::gated_pairs(bf16, R, E);
    auto product = [&](const char* name, long long lines, int stages, bool two) {
      const moe::GatedChoice c = moe::choose_gated(bf16, R, lines, stages, E, cus);
      std::printf("%s %s %d %d %d %d ", name, names[c.tile], c.splits, c.once, two, stages);
    };
    product("up", 2LL * p, sm, false);
    product("down", m, sp, pair);
    product("hidden", p, sm, false);
    product("x", m, 2 * sp, pair);
    const moe::GradWChoice w = moe::choose_grad_w(bf16, R, m, p, E, cus);
    std::printf("w %s %d 0 %d %d\n", w.wide ? "256x256x2" : "128x128x2", w.splits, pair, (R / E + steps - 1) / steps * (pair ? 2 : 1));
  }
  return 0;
}
