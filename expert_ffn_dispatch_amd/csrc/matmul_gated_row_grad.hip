// Gated projections, the rows' gradient: dgate W_gate + dup W_up.
#include "matmul_launch.h"

namespace moe {
hipError_t launch_matmul_gated_row_grad(const MatmulArgs& a, hipStream_t st) {
  return a.f16 ? launch_matmul_sizes<true, true, false, false, true>(a, st)
               : launch_matmul_sizes<false, true, false, false, true>(a, st);
}
}  // namespace moe
