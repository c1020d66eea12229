// Declarations between the launchers of the linear-attention passes.
#pragma once

#include <hip/hip_runtime_api.h>

#include "pdscan_linattn_plan.h"

namespace pdscan {

struct LaCarry {
  float* seg;            // contributions in, entering states out [segment][H]
  const float* decay;    // [segment][H]
  const float* user;     // state before the first segment in this direction [B][H], NULL: zero
  int rev;
};
struct LaCarryArgs {
  LaCarry c[2];
  const int32_t* starts; // packed: first segment of every sequence
  int B, H, nseg, tiles;   // tiles: workgroups of a state, 1024 elements each
  unsigned row;            // workgroups along x of the launch
  long long state;
};

hipError_t launch_linattn_form(const LaArgs& a, int bf16, int pass, hipStream_t st);
hipError_t launch_linattn_table(const int32_t* cu, int32_t* table, int32_t* starts, int B, int L, int seg, int segs,
                                hipStream_t st);
hipError_t launch_linattn_carry(const LaCarryArgs& a, int passes, hipStream_t st);
hipError_t launch_linattn_decay(const LaDecayArgs& a, hipStream_t st);
hipError_t launch_linattn_fold(const LaFoldArgs& a, hipStream_t st);
hipError_t launch_linattn_step(const LaStepArgs& a, hipStream_t st);

#define PDSCAN_LA_LAUNCHER(name) hipError_t name(const LaArgs& a, int nw, int pass, LaGrid g, hipStream_t st)
PDSCAN_LA_LAUNCHER(la_bf16_32);
PDSCAN_LA_LAUNCHER(la_bf16_64);
PDSCAN_LA_LAUNCHER(la_bf16_128);
PDSCAN_LA_LAUNCHER(la_bf16_256);
PDSCAN_LA_LAUNCHER(la_f32_32);
PDSCAN_LA_LAUNCHER(la_f32_64);
PDSCAN_LA_LAUNCHER(la_f32_128);
PDSCAN_LA_LAUNCHER(la_f32_256);

}  // namespace pdscan
