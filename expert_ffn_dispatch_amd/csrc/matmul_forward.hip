// Forward products: both operands hold the contraction contiguously.
#include "matmul_launch.h"

namespace moe {
hipError_t launch_matmul_forward(const MatmulArgs& a, hipStream_t st) {
  return a.f16 ? launch_matmul_form<true, true, true>(a, st) : launch_matmul_form<false, true, true>(a, st);
}
}  // namespace moe
