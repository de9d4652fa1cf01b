// Launches the tile kernel's instances of one form (one form per source file,
// so that they compile in parallel).
#pragma once
#include "matmul.h"
namespace moe {

template <bool F16, bool AKC, bool BKC, int BM, int BN, int WM, int WN, bool ALIGNED, bool EPI, bool GATED = false>
hipError_t launch_matmul_tile(const MatmulArgs& a, hipStream_t st) {
  constexpr bool WG = !AKC;
  const long long NT = ceil_div(a.n, GATED && AKC && BKC ? BN / 2 : BN);
  long long ub;                                   // at least the tiles of the list
  if (!WG && a.offsets != nullptr)
    ub = ((long long)a.rows / BM + (a.E < a.rows ? a.E : a.rows)) * NT;
  else
    ub = (long long)ceil_div(a.m, BM) * NT * (WG ? a.E : 1) + (long long)a.tail * (a.splits - 1);
  long long grid = (ub + 7) / 8 * 8;
  // Resident blocks walk the list; each loads its next tile's first stages
  // before it stores the last one.  Against one block per tile: 8192 x 4096 x
  // 16384 839 -> 823 us, 24576 rows over 160 experts of 1536 x 5120 659 -> 638.
  constexpr long long kResident = 256 * (BM * BN > 128 * 128 ? 1 : 2);
  if (grid > kResident) grid = kResident;
  if (grid <= 0) return hipSuccess;
  hipLaunchKernelGGL((matmul_tile_kernel<F16, AKC, BKC, BM, BN, WM, WN, ALIGNED, EPI, GATED>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, st, a);
  return hipGetLastError();
}

template <bool F16, bool AKC, bool BKC, bool EPI, bool GATED = false>
hipError_t launch_matmul_sizes(const MatmulArgs& a, hipStream_t st) {
  if (!a.aligned) return launch_matmul_tile<F16, AKC, BKC, 128, 128, 2, 2, false, EPI, GATED>(a, st);
  if (a.big) return launch_matmul_tile<F16, AKC, BKC, 256, 256, 2, 4, true, EPI, GATED>(a, st);
  return launch_matmul_tile<F16, AKC, BKC, 128, 128, 2, 2, true, EPI, GATED>(a, st);
}

template <bool F16, bool AKC, bool BKC>
hipError_t launch_matmul_form(const MatmulArgs& a, hipStream_t st) {
  if constexpr (AKC && BKC) {                     // gradients have nothing to apply
    if (a.bias != nullptr || a.pre != nullptr || a.act != kActNone || a.residual != nullptr)
      return launch_matmul_sizes<F16, AKC, BKC, true>(a, st);
  }
  return launch_matmul_sizes<F16, AKC, BKC, false>(a, st);
}

}  // namespace moe
