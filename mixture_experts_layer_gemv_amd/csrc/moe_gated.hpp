// Internal interface of the gated feed-forward block on plain weights and of
// the routing's gradient.  Every launch_* function only enqueues on the given
// stream; shapes are checked in moe_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// Widest m and p: the 32-bit offsets of a tile (256 lines of K or N values) fit.
constexpr int kGatedMaxCols = 1 << 20;

// One product over the experts' rows: out[r] = sum over K of x row r with the
// matrices of r's expert.
struct GatedArgs {
  const void* x;           // rows [..][K]
  const void* x2;          // second term's rows (gradient of x), or null
  const int32_t* perm;     // row r reads x row perm[r] / topk, or null (x row r)
  int T, topk;
  const void* w[2];        // the expert's matrices (gate and up; or one)
  const int32_t* offsets;  // [E+1] row ranges, or null (E = 1: all R rows)
  int R, E, K, N;          // rows, experts, reduction, output columns
  void* out[3];
  const void* in[2];       // gate, up [R][N] (gradient of the hidden rows)
  ptrdiff_t low;           // bytes from hidden rows to their low parts (gated_pairs), or 0: they have none
  float* part;             // workspace of a split reduction (gated_part_bytes), or null: none is split
};
// Whether R hidden rows of E experts are kept in two bf16 parts.
bool gated_low_parts(bool bf16, int R, int E);
// Bytes of `part` for a product of R rows with N output columns, by a reduction of K.
size_t gated_part_bytes(bool bf16, bool gated, int R, int K, int N, int E, int terms, int cus);

// The products with a weight gradient: out [E][M][N] = sum over an expert's
// rows r of x[r][i] w[r][j] (+ x2[r][i] w2[r][j]).
struct GradWProblem {
  const void* x;  // [R][M]
  const void* w;  // [R][N]
  const void *x2, *w2;  // the second term's, if an operand has a low part; else null
  void* out;
  int M, N;
};
struct GradWArgs {
  GradWProblem problem[3];
  int n;  // problems
  const int32_t* offsets;
  int R, E, m, p;  // m, p: of the block, whatever problems there are
  float* part;     // workspace of split reductions (grad_w_part_bytes), or null: none is split
};
size_t grad_w_part_bytes(bool bf16, int R, int m, int p, int E, int cus);

// bf16 or fp32 operands and outputs, fp32 sums.
//   gated_up:    out[0] = silu(x w0) * (x w1); out[1], out[2] = x w0, x w1 (or null)   w [E][K][N]
//   down:        out[0] = x w0                                                         w [E][K][N]
//   grad_hidden: dh = x w0^T; out[0], out[1] = gradients of gate and up, out[2] = h (or null)  w [E][N][K]
//   grad_x:      out[0] = x w0^T + x2 w1^T                                             w [E][N][K]
hipError_t launch_gated_up(const GatedArgs& a, bool bf16, int cus, hipStream_t s);
hipError_t launch_gated_down(const GatedArgs& a, bool bf16, int cus, hipStream_t s);
hipError_t launch_gated_grad_hidden(const GatedArgs& a, bool bf16, int cus, hipStream_t s);
hipError_t launch_gated_grad_x(const GatedArgs& a, bool bf16, int cus, hipStream_t s);
hipError_t launch_gated_grad_w(const GradWArgs& a, bool bf16, int cus, hipStream_t s);
// out[r] = x[perm[r] / topk], rows of `bytes` (a multiple of 16).
hipError_t launch_gather_rows(const void* x, const int32_t* perm, int T, int topk, int R, long long bytes, void* out,
                              hipStream_t s);

struct RouteGradArgs {
  const float* dw;        // [T][k] gradient of the gate weights
  const int32_t* idx;     // [T][k]
  const float* w;         // [T][k]
  const float* dl_add;    // [T][E] or null
  const void* x;          // [T][m]
  const float* wr;        // [m][E]
  const void* dx_add;     // [T][m] or null
  float* dl;              // [T][E]
  void* dx;               // [T][m] or null
  float* dwr;             // [m][E] or null
  float* db;              // [E] or null
  float* partial;         // workspace
  int T, m, E, k;
};
size_t route_grad_bytes(int T, int m, int E, int cus);
hipError_t launch_route_backward(const RouteGradArgs& a, bool bf16, int cus, hipStream_t s);

}  // namespace moe
