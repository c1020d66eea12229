// Instantiation of the product and state kernels of one type and x-row width,
// of those that a call can reach.
#pragma once

#include "pdscan_linattn.h"
#include "pdscan_linattn_launch.h"

namespace pdscan {

template <typename T, int DKP, int NW, int PASS>
hipError_t la_launch_pass(const LaArgs& a, LaGrid g, hipStream_t st) {
  using K = LaTile<T, DKP, NW>;
  if constexpr (la_reached(PASS, DKP, NW, !K::kF32)) {
    if constexpr (PASS == kLaPassState) {
      hipLaunchKernelGGL((pdssm_linattn_state_kernel<T, DKP, NW>), dim3(g.x, g.y), dim3(K::NT),
                         (unsigned)K::state_bytes(), st, a);
    } else {
      constexpr int QK = 1 << kLaQ | 1 << kLaK, V = 1 << kLaV;
      constexpr int JOBS = PASS == kLaPassFwd  ? 1 << kLaFwd
                           : PASS == kLaPassQK ? QK
                           : PASS == kLaPassV  ? V
                                               : QK | V;
      constexpr int NP = K::pieces(JOBS & QK ? kLaQ : kLaFwd);
      hipLaunchKernelGGL((pdssm_linattn_kernel<T, DKP, NW, JOBS>), dim3(g.x, g.y), dim3(K::NT),
                         (unsigned)K::main_bytes(NP), st, a);
    }
    return hipGetLastError();
  }
  return hipErrorInvalidValue;
}

template <typename T, int DKP, int NW>
hipError_t la_launch_nw(const LaArgs& a, int pass, LaGrid g, hipStream_t st) {
  return pass == kLaPassState ? la_launch_pass<T, DKP, NW, kLaPassState>(a, g, st)
         : pass == kLaPassFwd ? la_launch_pass<T, DKP, NW, kLaPassFwd>(a, g, st)
         : pass == kLaPassQK  ? la_launch_pass<T, DKP, NW, kLaPassQK>(a, g, st)
         : pass == kLaPassV   ? la_launch_pass<T, DKP, NW, kLaPassV>(a, g, st)
                              : la_launch_pass<T, DKP, NW, kLaPassQKV>(a, g, st);
}

template <typename T, int DKP>
hipError_t la_launch(const LaArgs& a, int nw, int pass, LaGrid g, hipStream_t st) {
  return nw == 1   ? la_launch_nw<T, DKP, 1>(a, pass, g, st)
         : nw == 2 ? la_launch_nw<T, DKP, 2>(a, pass, g, st)
                   : la_launch_nw<T, DKP, 4>(a, pass, g, st);
}

}  // namespace pdscan
