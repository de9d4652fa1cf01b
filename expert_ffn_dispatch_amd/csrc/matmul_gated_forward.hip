// Gated projections, forward: act(x W_gate^T) times x W_up^T.
#include "matmul_launch.h"

namespace moe {
hipError_t launch_matmul_gated_forward(const MatmulArgs& a, hipStream_t st) {
  return a.f16 ? launch_matmul_sizes<true, true, true, false, true>(a, st)
               : launch_matmul_sizes<false, true, true, false, true>(a, st);
}
}  // namespace moe
