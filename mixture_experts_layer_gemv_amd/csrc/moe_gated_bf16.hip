// The gated feed-forward block's products in bf16 (moe_gated_tile.hpp).
#include "moe_gated_tile.hpp"

namespace moe {

hipError_t gated_up_bf16(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<Bf16, Op::kUp>(a, cus, s); }
hipError_t gated_down_bf16(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<Bf16, Op::kDown>(a, cus, s); }
hipError_t gated_grad_hidden_bf16(const GatedArgs& a, int cus, hipStream_t s) {
  return rows_product<Bf16, Op::kGradHidden>(a, cus, s);
}
hipError_t gated_grad_x_bf16(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<Bf16, Op::kGradX>(a, cus, s); }
hipError_t gated_grad_w_bf16(const GradWArgs& a, int cus, hipStream_t s) { return grad_w_product<Bf16>(a, cus, s); }

}  // namespace moe
