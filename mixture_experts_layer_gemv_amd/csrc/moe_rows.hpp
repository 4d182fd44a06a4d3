// Internal interface of the row operators around the experts: the input
// norm's forward and backward pass, rows sorted into expert order and
// combined back with their gradients, and the int8 product.  Every launch_*
// function only enqueues on the given stream; shapes are checked in
// moe_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

struct NormArgs {
  const void* x;       // [T][m] bf16 or fp32
  const void* dy;      // backward: [T][m] in x's dtype
  const float* gamma;  // [m]
  const float* beta;   // [m] or null (forward, layer norm)
  void* out;           // forward: y [T][m]; backward: dx [T][m] or null
  float* mean;         // [T]: forward output or null, backward input (layer norm)
  float* rstd;         // [T]: forward output or null, backward input
  float* partial;      // backward with weight gradients: [2][blocks][m], or null
  float* dgamma;       // [m] or null
  float* dbeta;        // [m] or null
  float eps;
  int T, m;
  // with the residual's addition (add_norm):
  const void* residual;  // forward: [T][m] or null
  void* sum;             // forward: x + residual [T][m], or null
  int8_t* codes;         // forward: [T][m] or null
  float* scale;          // forward, with codes: [T]
  const void* dsum;      // backward: [T][m], added to dx, or null
};
hipError_t launch_norm_forward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s);
hipError_t launch_add_norm_forward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s);
hipError_t launch_add_norm_backward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s);

struct RowsArgs {
  const void* tok;     // token rows [T][m]: x (permute), dy (combine's gradient)
  const void* rows;    // expert rows [R][m]: input of the combine and of its gradient
  const int32_t* inv;  // [T*k] each assignment's expert row; outside [0, R): none
  const float* w;      // [T*k] gate weights, or null (all one)
  void* out;           // token rows (combine), expert rows (permute, combine's gradient) or null
  float* dw;           // [T*k] gradient of w, or null
  int T, m, k, R;
};
hipError_t launch_permute_rows(const RowsArgs& a, bool bf16, hipStream_t s);
hipError_t launch_combine_rows(const RowsArgs& a, bool rows_bf16, bool out_bf16, hipStream_t s);
hipError_t launch_combine_rows_backward(const RowsArgs& a, bool tok_bf16, bool rows_bf16, hipStream_t s);

// Longest reduction of the int8 product: 131071 * 128 * 128 < 2^31.
constexpr int kI8MaxK = 131056;

struct I8Args {
  const int8_t* x;         // [T][K] codes
  const float* sx;         // [T]
  const int8_t* w;         // [E][N][K] codes
  const float* sw;         // [E][N]
  const int32_t* offsets;  // [E+1] row ranges, or null (E = 1: all R rows)
  const int32_t* perm;     // [R]: row r reads x row perm[r] / topk, or null (x row r)
  void* y;                 // [R][N] bf16 or fp32
  int T, topk, R, K, N, E;
};
hipError_t launch_matmul_i8(const I8Args& a, bool y_bf16, int cus, hipStream_t s);

}  // namespace moe
