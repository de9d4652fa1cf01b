// Weight gradients: the contraction runs over the rows of both operands.
#include "matmul_launch.h"

namespace moe {
hipError_t launch_matmul_weight_grad(const MatmulArgs& a, hipStream_t st) {
  return a.f16 ? launch_matmul_form<true, false, false>(a, st) : launch_matmul_form<false, false, false>(a, st);
}
}  // namespace moe
