// Linear-attention products, fp32 inputs, x rows of up to 64 elements.
#include "pdscan_linattn_inst.h"

namespace pdscan {
hipError_t la_f32_64(const LaArgs& a, int nw, int pass, LaGrid g, hipStream_t st) {
  return la_launch<LaF32, 64>(a, nw, pass, g, st);
}
}  // namespace pdscan
