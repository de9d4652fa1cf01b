// Row gradients: dy holds the contraction contiguously, W has it as its rows.
#include "matmul_launch.h"

namespace moe {
hipError_t launch_matmul_row_grad(const MatmulArgs& a, hipStream_t st) {
  return a.f16 ? launch_matmul_form<true, true, false>(a, st) : launch_matmul_form<false, true, false>(a, st);
}
}  // namespace moe
