// The gated feed-forward block's products in fp32 (moe_gated_tile.hpp).
#include "moe_gated_tile.hpp"

namespace moe {

hipError_t gated_up_f32(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<F32, Op::kUp>(a, cus, s); }
hipError_t gated_down_f32(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<F32, Op::kDown>(a, cus, s); }
hipError_t gated_grad_hidden_f32(const GatedArgs& a, int cus, hipStream_t s) {
  return rows_product<F32, Op::kGradHidden>(a, cus, s);
}
hipError_t gated_grad_x_f32(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<F32, Op::kGradX>(a, cus, s); }
hipError_t gated_grad_w_f32(const GradWArgs& a, int cus, hipStream_t s) { return grad_w_product<F32>(a, cus, s); }

}  // namespace moe
