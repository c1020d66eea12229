// Instantiation of the product kernels of one type and x-row width.
#pragma once

#include "pdscan_linattn.h"
#include "pdscan_linattn_launch.h"

namespace pdscan {

template <typename T, int DKP, int NW>
hipError_t la_launch_nw(const LaArgs& a, int pieces, unsigned grid, hipStream_t st) {
  using K = LaTile<T, DKP, NW>;
  if (pieces == 0)
    hipLaunchKernelGGL((pdssm_linattn_state_kernel<T, DKP, NW>), dim3(grid), dim3(K::NT), (unsigned)K::state_bytes(),
                       st, a);
  else if (pieces == 2)
    hipLaunchKernelGGL((pdssm_linattn_kernel<T, DKP, NW, K::kF32 ? 1 : 2, false>), dim3(grid), dim3(K::NT),
                       (unsigned)K::main_bytes(K::kF32 ? 1 : 2), st, a);
  else
    hipLaunchKernelGGL((pdssm_linattn_kernel<T, DKP, NW, K::kF32 ? 1 : 3, true>), dim3(grid), dim3(K::NT),
                       (unsigned)K::main_bytes(K::kF32 ? 1 : 3), st, a);
  return hipGetLastError();
}

template <typename T, int DKP>
hipError_t la_launch(const LaArgs& a, int nw, int pieces, unsigned grid, hipStream_t st) {
  if constexpr (DKP < 256)
    if (nw == 1) return la_launch_nw<T, DKP, 1>(a, pieces, grid, st);
  if constexpr (DKP < 256 || !LaTile<T, DKP, 4>::kF32)
    if (nw == 2) return la_launch_nw<T, DKP, 2>(a, pieces, grid, st);
  return la_launch_nw<T, DKP, 4>(a, pieces, grid, st);
}

}  // namespace pdscan
