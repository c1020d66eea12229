// Stand-ins for the launchers and the error text of the linear-attention
// calls: programs on the host link the C ABI against them, so no call reaches
// a device.  Every launch is noted.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "pdscan.h"
#include "pdscan_error.h"
#include "pdscan_linattn_launch.h"

struct FormLaunch {
  int bf16, pass, DK, DV;
};
static std::vector<FormLaunch> g_forms;
static int g_launches = 0, g_fail = 0;

namespace pdscan {
int set_error(int code, const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  return code;
}
void clear_error() {}
hipError_t launch_linattn_form(const LaArgs& a, int bf16, int pass, hipStream_t) {
  ++g_launches;
  g_forms.push_back({bf16, pass, a.job[0].DK, a.job[0].DV});
  return hipSuccess;
}
hipError_t launch_linattn_table(const int32_t*, int32_t*, int32_t*, int, int, int, int, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_linattn_carry(const LaCarryArgs&, int, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_linattn_decay(const LaDecayArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_linattn_fold(const LaFoldArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_linattn_step(const LaStepArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
}  // namespace pdscan
extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }

static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::fprintf(stderr, "FAIL %s: status %d, expected %d\n", what, got, want);
    ++g_fail;
  }
}

static pdssm_linattn_dims dims(int B, int H, int Hk, int L, int dk, int dv, int packed = 0, int dtype = PDSSM_BF16) {
  pdssm_linattn_dims d;
  d.B = B; d.H = H; d.Hk = Hk; d.L = L; d.dk = dk; d.dv = dv;
  d.in_dtype = dtype; d.packed = packed; d.decay_per_head = 0; d.scale = 1.0f;
  return d;
}
