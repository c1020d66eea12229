// The kernels that the calls reach, by running the C ABI over every dk and dv
// of both types: one line each, "kernel<type, x row, waves, jobs>".
#include <set>
#include <string>

#include "linattn_stubs.h"

int main() {
  std::set<std::string> seen;
  for (int dtype : {PDSSM_F32, PDSSM_BF16})
    for (int dk = 8; dk <= 256; dk += 8)
      for (int dv = 8; dv <= 256; dv += 8)
        for (int L : {5, 4096}) {
          expect(call_fwd(dims(1, 1, 1, L, dk, dv, 0, dtype)), PDSSM_OK, "fwd");
          expect(call_bwd(dims(1, 1, 1, L, dk, dv, 0, dtype)), PDSSM_OK, "bwd");
        }
  for (const FormLaunch& f : g_forms) {
    const int jobs[] = {0, 1, 6, 8, 14};
    char text[64];
    const char* type = f.bf16 ? "LaBf16" : "LaF32";
    const int pad = pdscan::la_pad(f.DK), nw = pdscan::la_waves(f.DK, f.DV, f.bf16);
    if (f.pass == pdscan::kLaPassState)
      std::snprintf(text, sizeof text, "state_kernel<%s, %d, %d>", type, pad, nw);
    else
      std::snprintf(text, sizeof text, "kernel<%s, %d, %d, %d>", type, pad, nw, jobs[f.pass]);
    seen.insert(text);
    if (!pdscan::la_reached(f.pass, pad, nw, f.bf16)) ++g_fail;
  }
  for (const std::string& s : seen) std::printf("%s\n", s.c_str());
  std::printf("ok: %d failures, %d launches\n", g_fail, g_launches);
  return g_fail != 0;
}
