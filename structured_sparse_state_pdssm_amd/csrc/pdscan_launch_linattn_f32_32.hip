// Linear-attention products, fp32 inputs, x rows of up to 32 elements.
#include "pdscan_linattn_inst.h"

namespace pdscan {
hipError_t la_f32_32(const LaArgs& a, int nw, int pass, LaGrid g, hipStream_t st) {
  return la_launch<LaF32, 32>(a, nw, pass, g, st);
}
}  // namespace pdscan
