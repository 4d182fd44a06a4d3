// Index arithmetic of the row operators and the int8 product, shared by the
// kernels and a host test that checks it exhaustively.  No HIP dependency.
#pragma once

#include <stdint.h>

#include "moe_index.hpp"

namespace moe {

// ---- norm ------------------------------------------------------------------------

// Widest row: 1024 threads with two 8-element vectors.
constexpr int kNormMaxCols = 16384;

// The columns of vector v of thread tid in a team of NT threads, as two fours
// that start at lo and hi: eight together for bf16, twice four for fp32, so
// that a wave's 16-byte accesses always cover whole lines.
struct NormCols {
  int lo, hi;
};
MOE_HD inline NormCols norm_cols(bool bf16, int tid, int NT, int v) {
  if (bf16) return {8 * (tid + v * NT), 8 * (tid + v * NT) + 4};
  return {4 * (tid + 2 * v * NT), 4 * (tid + (2 * v + 1) * NT)};
}

// The same for a lane of a wave that takes 512 columns of a row: eights where
// all of the data is bf16, else twice four (fp32 rows, 8192 x 4096, top-2: the
// combine 64 -> 56 us, its gradient 118 -> 115).
MOE_HD inline NormCols slab_cols(bool fours, int lane, int slab) {
  const int at = 512 * slab;
  return fours ? NormCols{at + 4 * lane, at + 256 + 4 * lane} : NormCols{at + 8 * lane, at + 8 * lane + 4};
}

// Slabs of a row.  The combine's gradient walks them with up to four waves and
// two slabs a step: steps of 4096 columns, so that the columns past a row's end
// stay below 2^31 too.
MOE_HD inline int row_slabs(int m) { return (m - 1) / 512 + 1; }

// Vectors of 8 per thread, and threads of a team, for rows of m.
MOE_HD inline int norm_vecs(int m) { return m <= 8192 ? 1 : 2; }
MOE_HD inline int norm_threads(int m) {
  const int per = 8 * norm_vecs(m), n = (m + per - 1) / per;
  return n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : (n + 63) / 64 * 64;
}
// Teams of a block.
MOE_HD inline int norm_fwd_teams(int nt) { return nt <= 256 ? 256 / nt : 1; }
MOE_HD inline int norm_bwd_teams(int nt) { return nt <= 512 ? 512 / nt : 1; }

// So few steps that one block takes them all and no second launch is needed
// (rows of 4096: 4 steps 6.3 us, against 8.7 us for 5 on 5 blocks; 8192: 7.6
// us).  Rows past 8192 columns, without the next row loaded ahead, take 11 us.
constexpr int kNormOneBlockSteps = 4;

// Blocks of a backward pass, each of which writes a row of partial sums: one a
// CU (a second costs more partial sums than it hides: 4096 x 4096 fp32 38.0 and
// 39.7 us, 777 x 5000 13.4 and 15.4, 8192 x 4096 bf16 41.3 and 41.5), two where a
// row takes less than 256 threads (16384 x 1024 bf16: 24.4 and 23.6 us).
MOE_HD inline int norm_bwd_blocks(int T, int m, int cus) {
  const int nt = norm_threads(m), teams = norm_bwd_teams(nt);
  const long long steps = ((long long)T + teams - 1) / teams, most = (long long)cus * (nt < 256 ? 2 : 1);
  if (steps <= kNormOneBlockSteps && norm_vecs(m) == 1) return steps > 0;
  if (steps <= most) return (int)steps;
  const long long per = (steps + most - 1) / most;  // the same number of steps for every block but the last
  return (int)((steps + per - 1) / per);
}

// ---- int8 product ------------------------------------------------------------------

// A 128-byte line of a row r in LDS: its chunk c of 16 bytes is stored at place
// c ^ ((r >> 1) & 7).  Products read the same chunk of 16 successive rows in
// one LDS cycle (256 bytes): even rows lie in the lower and odd rows in the
// upper half of the banks, and the 8 rows of each half at 8 places, so no bank
// is read twice (r & 7 in its place: half of the LDS cycles were conflicts).
MOE_HD inline int line_place(int r, int c) { return c ^ ((r >> 1) & 7); }
// The copy of lines 8 i .. 8 i + 7 makes that order by the chunk that each lane
// fetches: lane l writes place l % 8 of line 8 i + l / 8.
MOE_HD inline int chunk_of(int i, int lane) { return (lane & 7) ^ ((4 * i + (lane >> 4)) & 7); }

// LDS byte of the 16 bytes a lane reads of 32 rows' quarter ks (32 bytes) of a
// stage, for 32 x 32 x 32 products (row lane % 32, chunk 2 ks + lane / 32), from
// the first row's line; and for 16 x 16 x 64 products, half ks of the stage
// (row lane % 16, chunk 4 ks + lane / 16).
MOE_HD inline int operand32(int lane, int ks) { return (lane & 31) * 128 + 16 * line_place(lane & 31, 2 * ks + (lane >> 5)); }
MOE_HD inline int operand16(int lane, int ks) { return (lane & 15) * 128 + 16 * line_place(lane & 15, 4 * ks + (lane >> 4)); }

// Stage s of [lo, hi) in a walk that begins rot stages (of less than hi - lo)
// further on.
MOE_HD inline int turned(int s, int rot, int lo, int hi) { return s + rot < hi ? s + rot : s + rot - (hi - lo); }

// A workgroup of WT x WC waves computes 32 TB WT rows by 32 CB WC channels with
// S stages of 128 bytes of the reduction in its ring.
template <int TB, int CB, int WT, int WC, int S>
struct TileShape {
  static constexpr int waves = WT * WC;
  static constexpr int BM = 32 * TB * WT, BN = 32 * CB * WC;
  static constexpr int XB = BM * 128, WB = BN * 128;  // bytes of a stage
  static constexpr int CPX = BM / 8 / waves, CPW = BN / 8 / waves, CP = CPX + CPW;  // copies per wave and stage
  static constexpr int RING = S * (XB + WB);
  // Waves a SIMD holds (of 4 a CU): one workgroup of eight waves, or as many of four as the LDS takes, up to two.
  static constexpr int per_simd = waves > 4 || 2 * RING <= 160 * 1024 ? 2 : 1;
  static_assert(BM % (8 * waves) == 0 && BN % (8 * waves) == 0, "every wave issues the same copies");
  static_assert(CP * (S - 1) <= 63, "vmcnt holds at most 63");
  // Epilogue: a wave stages 32 rows of its 32 CB channels of ES bytes, padded
  // by 16 bytes, and stores them 16 bytes a lane.
  static constexpr int row_bytes(int ES) { return 32 * CB * ES; }
  static constexpr int stride(int ES) { return row_bytes(ES) + 16; }
  static_assert(WT * WC * 32 * (32 * CB * 4 + 16) <= S * (32 * TB * WT + 32 * CB * WC) * 128, "the staging fits the ring");
};
// Element v of a 32 x 32 accumulator in a lane: its channel (of 32) in steps of
// four, the row being lane % 32.
MOE_HD inline int acc_channel(int lane, int v) { return 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3); }

// The kernels of the product, by their rows x channels x stages: tiles of a
// workgroup's waves, and (kRing) waves with rings of their own for few rows.
enum I8Kernel {
  kTile32x256x3,
  kTile64x256x3,
  kTile32x256x2,
  kTile64x256x2,
  kTile256x256x2,
  kTile128x256x3,
  kTile128x128x4,
  kTile64x128x3,
  kTile64x64x4,
  kRing16x32,
  kRing64x32,
  kRing32x32,
  kI8Kernels
};
// once: most experts' weights are read by one row block (tiles only; rings
// always start from different stages and look at each expert's blocks).  Then
// neighbouring tiles start from different stages, and large weights are not
// kept.  Its limits are a mean of three quarters of the 256-row block and of all
// of a smaller one.  Measured with once and without, weights from HBM (E * N * K
// of 600 MB or more in turn), 8 experts of so many rows in the mean: 256 x 256
// tiles, 4096 x 8192: 128 rows 61 and 78 us, 192 67 and 81, 224 75 and 84, 256 115
// and 121, 300 111 and 114; 256 dense rows, 8192 x 57344: 128 and 145; 128 x 128,
// 4096 x 4096: 96 rows 36 and 39, 128 50 and 51; 128 x 256, the same: 160 rows 42
// and 44; 64 x 128, 4096 x 3328: 40 rows 25 and 31, 64 37 and 40; 64 x 64: 70 dense
// rows, 16384 x 8192: 38.6 and 40.1.  So it still gains 2 to 12 % past the limits,
// which are on the low side.
struct I8Choice {
  I8Kernel kernel;
  bool once;
};

// The kernel for R >= 1 rows of E experts and N channels on `cus` CUs.
//
// The largest tile that still gives three quarters of the CUs an item, for
// experts of the mean row count: a tile reads (1 / BM + 1 / BN) bytes per
// product, but one round of too few tiles leaves CUs idle.  Half of the CUs
// are enough where the next smaller tile would need a second round.
inline I8Choice choose_i8(int R, int N, int E, int cus) {
  const long long experts = R < E ? R : E, avg = (R + experts - 1) / experts;
  auto items = [&](int BM, int BN) { return experts * ((avg + BM - 1) / BM) * ((N + BN - 1) / BN); };
  auto enough = [&](long long n, long long finer) { return 4 * n >= 3 * cus || (2 * n >= cus && finer > cus); };
  const long long n256 = items(256, 256), n128 = items(128, 256), n128s = items(128, 128);
  // Few rows, where most experts fit one row block of 32 or 64 (an even routing
  // spreads their counts by the square root of the mean, taken one and a half
  // times; a second block reads the weights again: 30 rows each of 8 experts,
  // 4096 x 14336: blocks of 32 109, of 64 76 us).  One workgroup a CU with a ring
  // of three stages where a round of them is five eighths full (16 x 4096 x
  // 49152, 192 items: 31.6, 64 x 64 39.6 us; 16 x 4096 x 32768, 128 items: 27.0
  // and 25.4), else two with two stages where the rounds are three quarters full
  // (16 rows each of 8 experts, 4096 x 14336, 448 items: 72 and 78 us; 7 rows each
  // of 64 experts, 1776 x 2464, 640 items: 75 and 62 us; 50 rows each of 8 experts,
  // 4096 x 14336: 79, 128 x 256 84 us).
  auto fit = [&](int BM) { return avg <= BM && (E == 1 || 4 * (BM - avg) * (BM - avg) >= 9 * avg); };
  const long long wide = experts * ((N + 255) / 256), round = 2LL * cus;
  if (wide <= cus && 8 * wide >= 5 * cus) {
    if (fit(32)) return {kTile32x256x3, true};
    if (fit(64)) return {kTile64x256x3, true};
  } else if (wide > cus && 3 * ((wide + round - 1) / round * round) <= 4 * wide) {
    if (fit(32)) return {kTile32x256x2, true};
    if (fit(64)) return {kTile64x256x2, true};
  }
  // 16384 rows of 8 experts, 4096 x 14336: 0.91, 128 x 256 1.05 ms; 128 rows each: 113 and 124 us;
  // 5565 x 2832 x 1680 (154 items, 308 of 128 x 256): 39 and 53 us
  if (avg > 112 && enough(n256, n128)) return {kTile256x256x2, avg <= 192};
  // 64 rows each of 8 experts: 89, 64 x 128 106 us; 2048 x 4096 x 4096 (128 items of 256 x 256): 37 and 43 us
  if (avg > 48 && enough(n128, n128s)) return {kTile128x256x3, avg <= 128};
  // 1003 x 6400 x 4096: 33 us, 128 x 256 40 us, 64 x 128 38 us
  if (avg > 64 && 4 * n128s >= 3 * cus) return {kTile128x128x4, avg <= 128};
  // 512 x 4096 x 4096: 16.1 us, 128 x 128 17.3 us
  if (avg > 32 && 4 * items(64, 128) >= 3 * cus) return {kTile64x128x3, avg <= 64};
  // 64 x 4096 x 14336: 12 us, 64 rows on private rings 16 us; 16 x 16384 x 16384: 40, 16 rows on them 45 us
  if (4 * items(64, 64) >= 3 * cus) return {kTile64x64x4, avg <= 64};
  // 16 x 14336 x 4096 (64 items of 64 channels): 11.4 us, 64 x 64 29 us
  if (avg <= 16) return {kRing16x32, true};
  // 64 x 8192 x 8192 (256 items of 32 channels): 14.6 us, 32 rows 21 us; 64 x 14336 x 4096 (128): 18.4 and 13.6 us
  if (avg > 32 && 4 * items(64, 32) >= 3 * cus) return {kRing64x32, true};
  // 64 x 14336 x 4096: 13.6 us, 64 x 64 29.5 us; a ring of one stage for eight waves in place of two for four 13.8 us
  // (64 x 8192 x 8192: 23 and 21 us)
  return {kRing32x32, true};
}

// Weights that their experts' only row block reads, too large for the 256 MB
// last-level cache to hold until the next call, are read as not to be kept:
// 16 rows each of 8 experts, 470 MB: 84 -> 72 us; 16 x 28672 x 8192: 41 -> 37 us;
// 184 MB between other calls 37 -> 32 us (alone and warm 28.6 -> 31 us); 58 MB,
// warm: 10.9 -> 12.5 us.  Rows that share lines (w off 128 bytes, or K) are
// fetched twice then (K = 1776, warm: 51 -> 62 us).
inline bool i8_weights_once(const void* w, int K, int N, int E) {
  return K % 128 == 0 && reinterpret_cast<uintptr_t>(w) % 128 == 0 && (long long)E * N * K >= 128 << 20;
}

}  // namespace moe
