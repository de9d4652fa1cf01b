// Gated projections, the weights' gradients: dgate^T x and dup^T x.
#include "matmul_launch.h"

namespace moe {
hipError_t launch_matmul_gated_weight_grad(const MatmulArgs& a, hipStream_t st) {
  return a.f16 ? launch_matmul_sizes<true, false, false, false, true>(a, st)
               : launch_matmul_sizes<false, false, false, false, true>(a, st);
}
}  // namespace moe
