// The work items of a launch over the experts' rows, found on the device from a
// dispatch's offsets; shared by the int8 product and the gated feed-forward
// block.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_gated_index.hpp"
#include "moe_index.hpp"

namespace moe {

// The value that the DPP control CTRL moves to each lane (0 where none does).
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_moved(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, true);
}
// Over the lanes up to each one (values >= 0): four shifts within rows of 16 lanes,
// then the rows' last values carried on.
__device__ __forceinline__ int scan_max(int v) {
  v = max(v, dpp_moved<0x111, 0xF>(v));  // row_shr:1
  v = max(v, dpp_moved<0x112, 0xF>(v));
  v = max(v, dpp_moved<0x114, 0xF>(v));
  v = max(v, dpp_moved<0x118, 0xF>(v));
  v = max(v, dpp_moved<0x142, 0xA>(v));         // row_bcast:15 into rows 1 and 3
  return max(v, dpp_moved<0x143, 0xC>(v));      // row_bcast:31 into rows 2 and 3
}
__device__ __forceinline__ int scan_sum(int v) {
  v += dpp_moved<0x111, 0xF>(v);
  v += dpp_moved<0x112, 0xF>(v);
  v += dpp_moved<0x114, 0xF>(v);
  v += dpp_moved<0x118, 0xF>(v);
  v += dpp_moved<0x142, 0xA>(v);
  return v + dpp_moved<0x143, 0xC>(v);
}

// One (expert, row block, column block) of a launch.
struct Item {
  int e, mb, nb;   // e < 0: none
  int blocks;      // row blocks of the expert
  int row0, rows;  // the block's first row and its rows
};

// Item L of the launch's work order (see gemm_item; cg = 0: row blocks
// outermost), found by every wave for itself: each lane holds an expert.  The
// offsets are clamped to [0, R], a decreasing entry counting as its
// predecessor, so that the ranges are disjoint and in bounds whatever the
// caller's array holds.  spread: L is the block's number, dealt evenly over
// the XCDs (xcd_item); else it is the item.  cut: see cut_last_round; the grid then
// has to hold cut_blocks blocks.
__device__ __forceinline__ Item find_item(const int32_t* offsets, int E, int R, int BM, int NBL, int cg, int L, bool spread,
                                          int cut = 0) {
  Item it{-1, 0, 0, 0, 0, 0};
  int half = -1;
  auto item_of = [&](int b, int total) {
    if (!spread) return b;
    const int last = cut ? cut_last_round(total, cut) : 0;
    if (!last) return xcd_item(b, total, 0);
    int i = xcd_item(b, total - last, 2 * last);
    if (i >= total - last) {
      half = (i - (total - last)) & 1;
      i = total - last + ((i - (total - last)) >> 1);
    }
    return i;
  };
  int e = 0, lo = 0, hi = R, before = 0;  // the item's expert, its rows, the items before it
  if (!offsets) {
    const int total = (hi + BM - 1) / BM * NBL;
    L = item_of(L, total);
    if (L < 0 || L >= total) return it;
  } else {
    const int lane = threadIdx.x & 63;
    auto clamped = [&](int i) { return min(max(i <= E ? offsets[i] : 0, 0), R); };
    const int first = scan_max(clamped(lane)), next = clamped(lane + 1);
    const int end = max(first, next);
    const int items = lane < E ? (end - first + BM - 1) / BM * NBL : 0;
    const int sum = scan_sum(items);  // of the experts up to this one
    const int total = __builtin_amdgcn_readlane(sum, 63);
    L = item_of(L, total);
    if (L < 0 || L >= total) return it;
    e = __builtin_ctzll(__ballot(L < sum));
    before = __builtin_amdgcn_readlane(sum - items, e);
    lo = __builtin_amdgcn_readlane(first, e);
    hi = __builtin_amdgcn_readlane(end, e);
  }
  const int blocks = (hi - lo + BM - 1) / BM, li = L - before;
  if (cg) {
    const int g = li / (blocks * cg), rem = li - g * blocks * cg;
    const int gw = min(NBL - g * cg, cg);
    it.mb = rem / gw;
    it.nb = g * cg + (rem - it.mb * gw);
  } else {
    it.mb = li / NBL;
    it.nb = li - it.mb * NBL;
  }
  it.e = e;
  it.blocks = blocks;
  it.row0 = lo + it.mb * BM;
  it.rows = min(BM, hi - it.row0);
  if (half >= 0) {
    it.row0 += half * (BM / 2);
    it.rows = half ? it.rows - BM / 2 : min(it.rows, BM / 2);
    if (it.rows <= 0) it.e = -1;
  }
  return it;
}

}  // namespace moe
