// The gated feed-forward block's products by type, and token rows copied into
// the experts' order for a weight gradient, whose reduction runs over them.
#include "moe_gated.hpp"

#include "moe_gated_index.hpp"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// One wave a row: out[r] = x[perm[r] / topk], 16 bytes a lane.
__global__ __launch_bounds__(256) void k_gather_rows(const u32x4_t* __restrict__ x, const int32_t* __restrict__ perm, int T,
                                                     int topk, int R, long long chunks, u32x4_t* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  for (long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); r < R; r += 4LL * gridDim.x) {
    int t = perm[r] / topk;
    t = t < 0 ? 0 : (t >= T ? T - 1 : t);
    const u32x4_t* src = x + (size_t)t * chunks;
    u32x4_t* dst = out + (size_t)r * chunks;
#pragma unroll 4
    for (long long c = lane; c < chunks; c += 64) dst[c] = src[c];
  }
}

}  // namespace

hipError_t launch_gather_rows(const void* x, const int32_t* perm, int T, int topk, int R, long long bytes, void* out,
                              hipStream_t s) {
  if (R <= 0) return hipSuccess;
  const long long blocks = ((long long)R + 3) / 4;
  k_gather_rows<<<(unsigned)(blocks < 1 << 22 ? blocks : 1 << 22), 256, 0, s>>>(
      static_cast<const u32x4_t*>(x), perm, T, topk, R, bytes / 16, static_cast<u32x4_t*>(out));
  return hipGetLastError();
}

bool gated_low_parts(bool bf16, int R, int E) { return gated_pairs(bf16, R, E); }

size_t gated_part_bytes(bool bf16, bool gated, int R, int K, int N, int E, int terms, int cus) {
  if (R <= 0) return 0;
  const long long lines = gated ? 2LL * N : N;
  const int steps = stage_steps(bf16 ? 2 : 4);
  const GatedChoice c = choose_gated(bf16, R, lines, (K + steps - 1) / steps * terms, E, cus);
  return c.splits > 1 ? (size_t)c.splits * R * lines * sizeof(float) : 0;
}

size_t grad_w_part_bytes(bool bf16, int R, int m, int p, int E, int cus) {
  const GradWChoice c = choose_grad_w(bf16, R, m, p, E, cus);
  return c.splits > 1 ? (size_t)c.splits * 3 * E * m * p * sizeof(float) : 0;
}

hipError_t gated_up_bf16(const GatedArgs& a, int cus, hipStream_t s);
hipError_t gated_up_f32(const GatedArgs& a, int cus, hipStream_t s);
hipError_t gated_down_bf16(const GatedArgs& a, int cus, hipStream_t s);
hipError_t gated_down_f32(const GatedArgs& a, int cus, hipStream_t s);
hipError_t gated_grad_hidden_bf16(const GatedArgs& a, int cus, hipStream_t s);
hipError_t gated_grad_hidden_f32(const GatedArgs& a, int cus, hipStream_t s);
hipError_t gated_grad_x_bf16(const GatedArgs& a, int cus, hipStream_t s);
hipError_t gated_grad_x_f32(const GatedArgs& a, int cus, hipStream_t s);
hipError_t gated_grad_w_bf16(const GradWArgs& a, int cus, hipStream_t s);
hipError_t gated_grad_w_f32(const GradWArgs& a, int cus, hipStream_t s);

namespace {
bool shapes_fit(const GatedArgs& a) {
  return a.K > 0 && a.K % 8 == 0 && a.K <= kGatedMaxCols && a.N > 0 && a.N % 8 == 0 && a.N <= kGatedMaxCols && a.E >= 1 &&
         a.E <= 64 && (a.offsets || a.E == 1);
}
}  // namespace

hipError_t launch_gated_up(const GatedArgs& a, bool bf16, int cus, hipStream_t s) {
  if (a.R <= 0) return hipSuccess;
  if (!shapes_fit(a)) return hipErrorInvalidValue;
  return bf16 ? gated_up_bf16(a, cus, s) : gated_up_f32(a, cus, s);
}
hipError_t launch_gated_down(const GatedArgs& a, bool bf16, int cus, hipStream_t s) {
  if (a.R <= 0) return hipSuccess;
  if (!shapes_fit(a)) return hipErrorInvalidValue;
  return bf16 ? gated_down_bf16(a, cus, s) : gated_down_f32(a, cus, s);
}
hipError_t launch_gated_grad_hidden(const GatedArgs& a, bool bf16, int cus, hipStream_t s) {
  if (a.R <= 0) return hipSuccess;
  if (!shapes_fit(a)) return hipErrorInvalidValue;
  return bf16 ? gated_grad_hidden_bf16(a, cus, s) : gated_grad_hidden_f32(a, cus, s);
}
hipError_t launch_gated_grad_x(const GatedArgs& a, bool bf16, int cus, hipStream_t s) {
  if (a.R <= 0) return hipSuccess;
  if (!shapes_fit(a)) return hipErrorInvalidValue;
  return bf16 ? gated_grad_x_bf16(a, cus, s) : gated_grad_x_f32(a, cus, s);
}
hipError_t launch_gated_grad_w(const GradWArgs& a, bool bf16, int cus, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  if (a.n > 3 || a.R < 0 || a.E < 1 || a.E > 64 || (!a.offsets && a.E != 1)) return hipErrorInvalidValue;
  for (int i = 0; i < a.n; ++i)
    if (a.problem[i].M <= 0 || a.problem[i].M % 8 || a.problem[i].M > kGatedMaxCols || a.problem[i].N <= 0 || a.problem[i].N % 8 || a.problem[i].N > kGatedMaxCols)
      return hipErrorInvalidValue;
  return bf16 ? gated_grad_w_bf16(a, cus, s) : gated_grad_w_f32(a, cus, s);
}

}  // namespace moe
