// Index arithmetic of the gated feed-forward block's products, shared by the
// kernels and a host test that checks it exhaustively.  No HIP dependency.
#pragma once

#include <stdint.h>

#include "moe_rows_index.hpp"

namespace moe {

// A stage is 128 bytes of every line of both operands: 64 reduction steps in
// bf16, 32 in fp32.  An operand whose reduction index is innermost in memory
// has a line per row: 128 bytes of that row (the int8 product's lines, see
// line_place, chunk_of and operand32).  One whose reduction index is outermost
// (weights [K][N], and both operands of a weight gradient) has a line per
// reduction step: 128 bytes of its columns, 64 in bf16, 32 in fp32; the lines of
// a column group follow one another, so an operand of B columns has B lines
// in either form.
constexpr int stage_steps(int es) { return 128 / es; }
// Column group and reduction step of line i.
MOE_HD inline int line_group(int i, int es) { return i / stage_steps(es); }
MOE_HD inline int line_step(int i, int es) { return i % stage_steps(es); }

// Chunk c (16 bytes) of reduction step k's line is stored at place c ^ 4 ((k >>
// 1) & 1): the transposing reads below take 64 bytes of four successive lines in
// one LDS cycle; lines of one parity share their half of the banks, and this
// puts them in different quarters.
MOE_HD inline int step_place(int k, int c) { return c ^ (((k >> 1) & 1) << 2); }
// The chunk that lane l of a copy of lines 8 j .. 8 j + 7 fetches (line 8 j + l / 8).
MOE_HD inline int step_chunk(int lane) { return (lane & 7) ^ (((lane >> 4) & 1) << 2); }

// LDS byte, from the column group's first line, of the 8 bytes that a lane gives
// to transposing read t (0 or 1) of 32 columns (half 0 or 1 of the group's 64),
// quarter ks of a stage, bf16.  The read hands lane l of 16 the l-th column of
// four lines, lanes 4 q .. 4 q + 3 pointing at line q: after both reads a lane
// holds steps 16 ks + 8 (lane / 32) + 0 .. 7 of column lane % 32.
MOE_HD inline int transposed_read(int lane, int half, int ks, int t) {
  const int k = 16 * ks + 8 * (lane >> 5) + 4 * t + ((lane & 15) >> 2);
  const int c = 4 * half + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  return k * 128 + 16 * step_place(k, c) + 8 * (lane & 1);
}
// fp32: byte of step 8 ks + 4 (lane / 32) + i of column lane % 32 of a group.  A read of
// 4 bytes a lane takes 32 lanes a cycle, 32 columns of one line: no bank twice (333 tokens,
// top-3 of 12, 1000 x 1720: 5.3 M LDS cycles, which two a read account for, 2 % of them
// conflicts).
MOE_HD inline int step_read_f32(int lane, int ks, int i) {
  const int k = 8 * ks + 4 * (lane >> 5) + i;
  return k * 128 + 16 * step_place(k, (lane & 31) >> 2) + 4 * (lane & 3);
}

// Block b's expert and tile (of `tiles` of every expert) in a launch of 8
// ceil(tiles / 8) E blocks; e >= E: none.  Every XCD (b % 8) takes an eighth of each
// expert's tiles, one expert after the other: the experts' reductions differ in
// length, so an XCD that took whole experts would end before the others (16 experts
// of 410 to 1640 rows, three gradients of 4096 x 6400: 4.24 ms, so 2.43).
struct ExpertItem {
  int e, tile;
};
MOE_HD inline ExpertItem expert_item(int b, int tiles) {
  const int x = b & 7, j = b >> 3;
  const int lo = (int)((long long)x * tiles / 8), mine = (int)((long long)(x + 1) * tiles / 8) - lo;
  if (!mine) return {1 << 30, 0};
  return {j / mine, lo + j % mine};
}

// Items of the last round of `total` equal ones on `cus` CUs, if it would leave half
// of them idle or more: these are cut into two of half the rows each.  16384 rows of 8
// experts, 14336 x 4096 (1152 items, 4.5 rounds): 1.85 -> 1.73 ms; their gradient, 16
// experts, 2 x 6400 x 4096: 1.68 -> 1.58 ms.  Of many rounds the last one costs less
// than its cut items' second copies of the weights (8064 items: 3.28 and 3.32 ms).
MOE_HD inline int cut_last_round(int total, int cus) {
  const int last = total % cus;
  return total > cus && total <= 16 * cus && 2 * last <= cus ? last : 0;
}
// Blocks of a launch of at most `most` items that may be so cut.
inline long long cut_blocks(long long most, int cus) { return (most + cus / 2 + 7) / 8 * 8 + 16; }

// The 32-channel block of a tile's W lines that a wave's block c is.  Gated tiles
// hold their gate channels in the first half of the lines and the same channels
// of up in the second, and a wave takes both of each: c < CB / 2 is gate.
MOE_HD inline int channel_block(bool gated, int WC, int CB, int wc, int c) {
  if (!gated) return wc * CB + c;
  const int h = CB / 2;
  return c < h ? wc * h + c : WC * h + wc * h + (c - h);
}

// The tiles of the products over the experts' rows, by rows x weight lines x stages
// (a gated tile's lines are half gate, half up).
enum GatedTile {
  kGated256x256x2,
  kGated128x256x3,
  kGated128x128x2,
  kGated64x128x3,
  kGated32x256x2,
  kGated32x256x3,
  kGated32x128x2,
  kGatedTiles
};

// A product's tile; the number of blocks that share a tile's reduction, each of them
// some of its stages (their partial sums are joined by a second launch); and
// whether the weights are read as not to be kept in the caches.
struct GatedChoice {
  GatedTile tile;
  int splits;
  bool once;
};

// Hidden rows of so few rows an expert are handed to the next product in two bf16
// parts, 16 bits of each value: their products cost nothing there, where the weights'
// bytes bound the time (1 token 125 us with and without), and the outputs are as
// good as rounded once.
inline bool gated_pairs(bool bf16, int R, int E) {
  const long long experts = R < E ? R : E;
  return bf16 && R > 0 && (R + experts - 1) / experts <= 32;
}

// The choice for R >= 1 rows of E experts, `lines` weight lines (output columns,
// twice that for gate and up) and `stages` stages of all terms on `cus` CUs.
inline GatedChoice choose_gated(bool bf16, int R, long long lines, int stages, int E, int cus) {
  const long long experts = R < E ? R : E, avg = (R + experts - 1) / experts;
  auto items = [&](int BM, int BN) { return experts * ((avg + BM - 1) / BM) * ((lines + BN - 1) / BN); };
  GatedTile tile;
  long long n, slots = cus;  // tiles, and those that run at once
  if (bf16) {
    // 256 rows each of 8 experts, 4096 x 14336: gate and up 0.62, 128 x 256 0.69 ms (down 0.36 and 0.43)
    if (avg > 112 && 4 * items(256, 256) >= 3 * cus) tile = kGated256x256x2, n = items(256, 256);
    // 64 rows each of 8: 0.40, 256 x 256 0.47, 64 x 128 0.44 ms
    else if (avg > 64 && 4 * items(128, 256) >= 3 * cus) tile = kGated128x256x3, n = items(128, 256);
    // 83 rows each of 12, 1000 x 1720: down 27 (split in 2), 256 x 256 48, 64 x 128 24 us
    else if (avg > 64) tile = kGated128x128x2, n = items(128, 128), slots = 2 * cus;
    else if (avg > 32) tile = kGated64x128x3, n = items(64, 128), slots = 2 * cus;
    // 8 rows each of 16, 4096 x 6400, 800 tiles: gate and up 273, with one block a CU and three stages 291 us
    else if (items(32, 256) > cus) tile = kGated32x256x2, n = items(32, 256), slots = 2 * cus;
    // one row of 2 experts, 4096 x 14336, 224 tiles: 82, with two stages 98 us
    else tile = kGated32x256x3, n = items(32, 256);
  } else {
    // fp32's products take eight times as long, so it is their count that matters,
    // rows past an expert's last among it: 83 rows each of 12, 1000 x 1720: gate and up
    // 82, 128 x 128 131, 64 x 128 118 us; and every CU needs a share of them.
    auto fills = [&](int BM) {
      const long long tiles = items(BM, 128), most = 2 * cus / tiles, shares = most < stages / 4 ? most : stages / 4;
      return 4 * tiles * (shares > 1 ? shares : 1) >= 6 * cus;
    };
    // 4096 x 2048 x 8192: 1.02 ms (135 TFLOP/s), 64 x 128 1.10
    if (avg > 512 && fills(128)) tile = kGated128x128x2, n = items(128, 128), slots = 2 * cus;
    // 207 rows each of 5, 1000 x 712: hidden gradients 35, 128 x 128 47, 32 x 128 41 us (all split)
    else if (avg > 112 && fills(64)) tile = kGated64x128x3, n = items(64, 128), slots = 2 * cus;
    else tile = kGated32x128x2, n = items(32, 128), slots = 4 * cus;
  }
  // Too few tiles to fill the CUs share their reductions, at least four stages each:
  // one row of 2 experts, 14336 x 4096: 52 with the join, unsplit 144 us; 2 rows of 512 x 1024 in fp32: 16 and 45 us.
  // Short ones in bf16 do not pay for the join (512 to 1024 wide, one row: 12.1 and 11.3
  // us; 300 rows each of 4, 640 x 768: 33 and 25 us the pass; one row of 960: 22 and 26).
  long long splits = slots / n;
  if (splits > stages / 4) splits = stages / 4;
  if (splits > 32) splits = 32;
  if (bf16 && stages < (avg > 32 ? 16 : 10)) splits = 1;
  // Weights that few rows read, too large for the 256 MB last-level cache to hold until
  // the next call: 8 rows each of 16, 1.7 GB: 292 -> 273 us; one of 2, 470 MB: 88 -> 82 us.
  // Small ones, warm: 17.8 -> 21.4 us (1024 x 2048).  The mean decides, since the host does not
  // know the counts.  An expert that takes more rows than the mean has several row blocks, which
  // read its weights at the same time, most of them from the L2: gate and up of 512 rows, 16
  // experts, 4096 x 6400, a half of the rows for one expert: 417 and, kept, 423 us (even counts
  // 292 and 307), 2048 rows, 64 experts, 2048 x 1408: 194 and 196 (160 and 170).  Only where one
  // expert takes all rows, and its weights alone would fit the cache, does it lose: 198 and
  // 146, 90 and 55 us.
  const bool once = bf16 && avg <= 32 && (long long)experts * lines * stages * 128 >= 128LL << 20;
  return {tile, splits < 2 ? 1 : (int)splits, once};
}

// The weight gradients of R rows of E experts (two of m x p, one of p x m): 256 x 256
// tiles, or else 128 x 128, and the number of blocks that share a tile's rows.
struct GradWChoice {
  bool wide;
  int splits;
};
inline GradWChoice choose_grad_w(bool bf16, int R, int m, int p, int E, int cus) {
  auto tiles = [&](int B) { return 3LL * E * ((m + B - 1) / B) * ((p + B - 1) / B); };
  // 16 experts, 4096 x 6400: 2.4 ms with 256 x 256 tiles.  With fewer than two a CU, or
  // in fp32: 207 rows each of 5, 1000 x 712 in fp32: 85 -> 62 us.  So few that CUs idle share
  // their rows: 1134 rows of 432 x 560 in fp32: 70 -> 37 us.
  if (bf16 && tiles(256) >= 2 * cus) return {true, 1};
  const int steps = stage_steps(bf16 ? 2 : 4);
  const long long stages = (R / E + steps - 1) / steps;
  long long splits = 2 * cus / tiles(128);
  if (splits > stages / 4) splits = stages / 4;
  return {false, splits < 2 ? 1 : splits > 32 ? 32 : (int)splits};
}

}  // namespace moe
