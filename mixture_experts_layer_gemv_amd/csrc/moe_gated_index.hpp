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
// fp32: byte of step 8 ks + 4 (lane / 32) + i of column lane % 32 of a group.
MOE_HD inline int step_read_f32(int lane, int ks, int i) {
  const int k = 8 * ks + 4 * (lane >> 5) + i;
  return k * 128 + 16 * step_place(k, (lane & 31) >> 2) + 4 * (lane & 3);
}

// The 32-channel block of a tile's W lines that a wave's block c is.  Gated tiles
// hold their gate channels in the first half of the lines and the same channels
// of up in the second, and a wave takes both of each: c < CB / 2 is gate.
MOE_HD inline int channel_block(bool gated, int WC, int CB, int wc, int c) {
  if (!gated) return wc * CB + c;
  const int h = CB / 2;
  return c < h ? wc * h + c : WC * h + wc * h + (c - h);
}

}  // namespace moe
