// Checks the index arithmetic of the gated feed-forward block's products
// (moe_gated_index.hpp) on the host: the LDS places of both kinds of lines, the
// operand reads against a model of the buffers and of the transposing read, and
// the channel blocks of the waves.
#include <cstdio>
#include <set>
#include <vector>

#include "moe_gated_index.hpp"

static int fails = 0;
#define CHECK(c, ...)                                     \
  do {                                                    \
    if (!(c)) {                                           \
      if (fails++ < 20) {                                 \
        std::printf("line %d: %s: ", __LINE__, #c);       \
        std::printf(__VA_ARGS__);                         \
        std::printf("\n");                                \
      }                                                   \
    }                                                     \
  } while (0)

// An operand of `lines` lines with the reduction index outermost: every 8 bytes
// of LDS hold (step, first column) of the values that the copies bring there.
struct Half {
  int step, col;
};
static std::vector<Half> copied(int lines, int es) {
  std::vector<Half> lds(lines * 16, Half{-1, -1});
  for (int j = 0; j < lines / 8; ++j)
    for (int l = 0; l < 64; ++l) {
      const int i = 8 * j + l / 8, k = moe::line_step(i, es), g = moe::line_group(i, es);
      CHECK(k == (i % moe::stage_steps(es)) && (moe::step_place(k, moe::step_chunk(l)) == (l & 7)), "line %d lane %d", i, l);
      for (int h = 0; h < 2; ++h)
        lds.at((j * 64 + l) * 2 + h) = Half{k, (g * 128 + 16 * moe::step_chunk(l) + 8 * h) / es};
    }
  return lds;
}

static void bf16(int columns) {
  const std::vector<Half> lds = copied(columns, 2);
  for (int block = 0; block < columns / 32; ++block)
    for (int ks = 0; ks < 4; ++ks)
      for (int t = 0; t < 2; ++t) {
        // the read of a lane, as the kernels form it
        auto at = [&](int l) {
          const int a = (block >> 1) * 8192 + (moe::transposed_read(l, 0, 0, 0) ^ ((block & 1) << 6)) + ks * 2048 + t * 512;
          CHECK(a == (block >> 1) * 8192 + moe::transposed_read(l, block & 1, ks, t), "lane %d block %d", l, block);
          CHECK(a % 8 == 0 && a >= 0 && a + 8 <= columns * 128, "lane %d", l);
          return a;
        };
        for (int l = 0; l < 64; ++l)
          for (int q = 0; q < 4; ++q) {
            // element q of lane l comes from lane 4 q + (l % 16) / 4 of its sixteen, element l % 4
            const Half& h = lds.at(at((l & ~15) + 4 * q + ((l & 15) >> 2)) / 8);
            const int col = h.col + (l & 3), want = 32 * block + (l & 31);
            CHECK(col == want && h.step == 16 * ks + 8 * (l >> 5) + 4 * t + q, "block %d ks %d t %d lane %d: column %d step %d",
                  block, ks, t, l, col, h.step);
          }
        for (int half = 0; half < 2; ++half) {  // 32 lanes of 8 bytes: all 64 banks once
          std::set<int> banks;
          for (int l = 32 * half; l < 32 * half + 32; ++l) banks.insert(at(l) / 8 % 32);
          CHECK(banks.size() == 32, "block %d ks %d: %zu of 32", block, ks, banks.size());
        }
      }
}

static void fp32(int columns) {
  const std::vector<Half> lds = copied(columns, 4);
  for (int block = 0; block < columns / 32; ++block)
    for (int ks = 0; ks < 4; ++ks)
      for (int i = 0; i < 4; ++i)
        for (int l = 0; l < 64; ++l) {
          const int a = block * 4096 + moe::step_read_f32(l, ks, i);
          CHECK(a % 4 == 0 && a + 4 <= columns * 128, "lane %d", l);
          const Half& h = lds.at(a / 8);
          CHECK(h.col + a % 8 / 4 == 32 * block + (l & 31) && h.step == 8 * ks + 4 * (l >> 5) + i, "block %d ks %d i %d lane %d",
                block, ks, i, l);
        }
}

// Rows with the reduction innermost: a lane's 16 bytes are steps that match the
// other form's (8 in bf16, 4 in fp32 from the same first one).
static void rows() {
  for (int ks = 0; ks < 4; ++ks)
    for (int l = 0; l < 64; ++l) {
      const int a = moe::operand32(l, ks), r = a / 128, place = a % 128 / 16;
      int chunk = -1;
      for (int c = 0; c < 8; ++c)
        if (moe::line_place(r, c) == place) chunk = c;
      CHECK(r == (l & 31) && chunk * 16 / 2 == 16 * ks + 8 * (l >> 5) && chunk * 16 / 4 == 8 * ks + 4 * (l >> 5), "lane %d", l);
    }
}

static void channels(int WC, int CB) {
  for (int gated = 0; gated < 2; ++gated) {
    std::set<int> seen;
    for (int wc = 0; wc < WC; ++wc)
      for (int c = 0; c < CB; ++c) {
        const int b = moe::channel_block(gated, WC, CB, wc, c);
        CHECK(b >= 0 && b < WC * CB && seen.insert(b).second, "wave %d block %d", wc, c);
        // a gated wave's blocks: its channels of gate, the same of up half the tile later
        if (gated && c >= CB / 2) CHECK(b == moe::channel_block(true, WC, CB, wc, c - CB / 2) + WC * CB / 2, "wave %d", wc);
      }
  }
}

// Every (expert, tile) exactly once, and an XCD's experts in order.
static void items(int E, int tiles) {
  std::set<std::pair<int, int>> seen;
  int before[8] = {};
  for (int b = 0; b < 8 * ((tiles + 7) / 8) * E; ++b) {
    const moe::ExpertItem it = moe::expert_item(b, tiles);
    if (it.e >= E) continue;
    CHECK(it.e >= before[b & 7] && it.tile >= 0 && it.tile < tiles && seen.insert({it.e, it.tile}).second, "block %d", b);
    before[b & 7] = it.e;
  }
  CHECK((int)seen.size() == E * tiles, "%zu of %d x %d", seen.size(), E, tiles);
}

// Items of which the last round's are cut in two: each whole item once, each half once,
// within the blocks that the launch holds.
static void cut(int most, int total, int cus) {
  const int last = moe::cut_last_round(total, cus);
  CHECK(last >= 0 && last < cus && (!last || 2 * last <= cus), "%d", last);
  std::vector<int> seen(total + last, 0);
  const long long blocks = moe::cut_blocks(most, cus);
  CHECK(blocks % 8 == 0, "%lld", blocks);
  for (long long b = 0; b < blocks; ++b) {
    const int i = last ? moe::xcd_item((int)b, total - last, 2 * last) : moe::xcd_item((int)b, total, 0);
    if (i < 0) continue;
    CHECK(i < total + last, "block %lld item %d", b, i);
    if (i < total + last) seen[i]++;
  }
  for (int i = 0; i < total + last; ++i) CHECK(seen[i] == 1, "item %d of %d (%d cut): %d", i, total, last, seen[i]);
}

int main() {
  for (int total : {1, 7, 255, 256, 257, 300, 383, 384, 385, 511, 513, 1152, 1153, 1800, 4096, 4097, 5000})
    for (int more : {0, 1, 9, 100}) {
      cut(total + more, total, 256);
      cut(total + more, total, 304);
    }
  for (int E : {1, 2, 16, 64})
    for (int tiles : {1, 3, 7, 8, 9, 100, 1201}) items(E, tiles);
  for (int columns : {64, 128, 256}) {
    bf16(columns);
    fp32(columns);
  }
  rows();
  for (int WC : {1, 2, 4})
    for (int CB : {2, 4}) channels(WC, CB);
  if (fails) {
    std::printf("%d failures\n", fails);
    return 1;
  }
  std::printf("gated index check ok\n");
  return 0;
}
