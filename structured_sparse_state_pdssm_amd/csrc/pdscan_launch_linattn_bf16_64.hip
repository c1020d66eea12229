// Linear-attention products, bf16 inputs, x rows of up to 64 elements.
#include "pdscan_linattn_inst.h"

namespace pdscan {
hipError_t la_bf16_64(const LaArgs& a, int nw, int pass, LaGrid g, hipStream_t st) {
  return la_launch<LaBf16, 64>(a, nw, pass, g, st);
}
}  // namespace pdscan
