// The gated feed-forward block's products in bf16 (moe_gated_tile.hpp).
#include "moe_gated_tile.hpp"

namespace moe {
namespace {
constexpr int kGroup = 4;  // column blocks that share their rows in an XCD's L2

template <Op OP>
hipError_t rows_product(const GatedArgs& a, int cus, hipStream_t s) {
  const long long experts = a.R < a.E ? a.R : a.E, avg = (a.R + experts - 1) / experts;
  if (avg > 64) return launch_tile<Bf16, OP, 4, 2, 2, 4, 2>(a, kGroup, s);
  return launch_tile<Bf16, OP, 1, 2, 2, 4, 3>(a, kGroup, s);
}
}  // namespace

hipError_t gated_up_bf16(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<Op::kUp>(a, cus, s); }
hipError_t gated_down_bf16(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<Op::kDown>(a, cus, s); }
hipError_t gated_grad_hidden_bf16(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<Op::kGradHidden>(a, cus, s); }
hipError_t gated_grad_x_bf16(const GatedArgs& a, int cus, hipStream_t s) { return rows_product<Op::kGradX>(a, cus, s); }
hipError_t gated_grad_w_bf16(const GradWArgs& a, int, hipStream_t s) { return launch_grad_w_tile<Bf16, 4, 2, 2, 4, 2>(a, kGroup, s); }

}  // namespace moe
