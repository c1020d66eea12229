// Instantiation of the product kernels of one type and x-row width.
#pragma once

#include "pdscan_linattn.h"
#include "pdscan_linattn_launch.h"

namespace pdscan {

template <typename T, int DKP, int NW>
hipError_t la_launch_nw(const LaArgs& a, int pass, LaGrid g, hipStream_t st) {
  using K = LaTile<T, DKP, NW>;
  const unsigned two = (unsigned)K::main_bytes(K::pieces(kLaFwd)), three = (unsigned)K::main_bytes(K::pieces(kLaQ));
  constexpr int F = 1 << kLaFwd, Q = 1 << kLaQ | 1 << kLaK, V = 1 << kLaV;
  if (pass == kLaPassState)
    hipLaunchKernelGGL((pdssm_linattn_state_kernel<T, DKP, NW>), dim3(g.x, g.y), dim3(K::NT), (unsigned)K::state_bytes(),
                       st, a);
  else if (pass == kLaPassFwd)
    hipLaunchKernelGGL((pdssm_linattn_kernel<T, DKP, NW, F>), dim3(g.x, g.y), dim3(K::NT), two, st, a);
  else if (pass == kLaPassQK)
    hipLaunchKernelGGL((pdssm_linattn_kernel<T, DKP, NW, Q>), dim3(g.x, g.y), dim3(K::NT), three, st, a);
  else if (pass == kLaPassV)
    hipLaunchKernelGGL((pdssm_linattn_kernel<T, DKP, NW, V>), dim3(g.x, g.y), dim3(K::NT), two, st, a);
  else
    hipLaunchKernelGGL((pdssm_linattn_kernel<T, DKP, NW, Q | V>), dim3(g.x, g.y), dim3(K::NT), three, st, a);
  return hipGetLastError();
}

template <typename T, int DKP>
hipError_t la_launch(const LaArgs& a, int nw, int pass, LaGrid g, hipStream_t st) {
  if constexpr (DKP < 256)
    if (nw == 1) return la_launch_nw<T, DKP, 1>(a, pass, g, st);
  if constexpr (DKP < 256 || !LaTile<T, DKP, 4>::kF32)
    if (nw == 2) return la_launch_nw<T, DKP, 2>(a, pass, g, st);
  return la_launch_nw<T, DKP, 4>(a, pass, g, st);
}

}  // namespace pdscan
