// Index arithmetic of the row operators and the int8 product, shared by the
// kernels and a host test that checks it exhaustively.  No HIP dependency.
#pragma once

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

}  // namespace moe
