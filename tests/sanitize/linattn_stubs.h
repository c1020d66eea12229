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
// What the device takes: fewer than 2^32 threads along an axis, 65535 rows, and
// every workgroup numbered in 31 bits.
inline void launch_of(long long blocks, int threads) {
  ++g_launches;
  const LaGrid g = la_grid_rows(blocks, threads);
  const long long all = (long long)g.x * g.y;
  if (blocks < 1 || blocks > 0x7fffffffll || (long long)g.x * threads > 0xffffffffll || g.y > 65535 || all < blocks ||
      all - blocks >= g.y) {
    std::fprintf(stderr, "FAIL a launch of %lld x %d threads\n", blocks, threads);
    ++g_fail;
  }
}
hipError_t launch_linattn_form(const LaArgs& a, int bf16, int pass, hipStream_t) {
  launch_of(la_grid(a), 64 * la_waves(a.job[0].DK, a.job[0].DV, bf16));
  g_forms.push_back({bf16, pass, a.job[0].DK, a.job[0].DV});
  return hipSuccess;
}
hipError_t launch_linattn_table(const int32_t*, int32_t*, int32_t*, int, int, int, int, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_linattn_carry(const LaCarryArgs& a, int, hipStream_t) { launch_of((long long)a.B * a.H, 256); if (a.tiles != (a.state / 4 + 255) / 256) ++g_fail; return hipSuccess; }
hipError_t launch_linattn_decay(const LaDecayArgs& a, hipStream_t) { launch_of((long long)a.c.segs * a.c.H, kLaPiece); return hipSuccess; }
hipError_t launch_linattn_fold(const LaFoldArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_linattn_step(const LaStepArgs& a, hipStream_t) {
  launch_of((long long)a.B * a.H * ((a.dv + a.cols - 1) / a.cols), 256);
  return hipSuccess;
}
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

static void* at(int slot) { return (void*)(uintptr_t)(0x100000000000ull + ((uint64_t)slot << 50)); }

static pdssm_view view(int slot, const pdssm_linattn_dims& d, int heads, int width) {
  pdssm_view v;
  v.data = at(slot);
  v.stride_t = width;
  v.stride_h = (int64_t)d.L * width;
  v.stride_b = (int64_t)heads * d.L * width;
  return v;
}

// The calls on fake addresses; the statuses of a query and its call agree.
static int call_fwd(const pdssm_linattn_dims& d) {
  pdssm_view q = view(0, d, d.Hk, d.dk), k = view(1, d, d.Hk, d.dk), v = view(2, d, d.H, d.dv), o = view(3, d, d.H, d.dv),
             g = view(4, d, d.H, 1);
  size_t n = 0;
  const int rc = pdssm_linattn_workspace_bytes(&d, &n);
  const int rd = pdssm_linattn_fwd(&d, &q, &k, &v, &g, d.packed ? (const int32_t*)at(5) : nullptr, (float*)at(6), &o,
                                   (float*)at(7), at(8), n, nullptr);
  expect(rd, rc, "query and call");
  return rd;
}
static int call_bwd(const pdssm_linattn_dims& d) {
  pdssm_view q = view(0, d, d.Hk, d.dk), k = view(1, d, d.Hk, d.dk), v = view(2, d, d.H, d.dv), o = view(3, d, d.H, d.dv),
             g = view(4, d, d.H, 1);
  pdssm_view gq = view(5, d, d.Hk, d.dk), gk = view(6, d, d.Hk, d.dk), gv = view(7, d, d.H, d.dv), gg = view(8, d, d.H, 1);
  size_t n = 0;
  const int rc = pdssm_linattn_bwd_workspace_bytes(&d, &n);
  const int rd = pdssm_linattn_bwd(&d, &q, &k, &v, &g, d.packed ? (const int32_t*)at(9) : nullptr, (float*)at(10), &o,
                                   (float*)at(11), &gq, &gk, &gv, &gg, (float*)at(12), at(13), n, nullptr);
  expect(rd, rc, "gradient's query and call");
  return rd;
}
static int call_step(const pdssm_linattn_dims& d) {
  pdssm_view q = view(0, d, d.Hk, d.dk), k = view(1, d, d.Hk, d.dk), v = view(2, d, d.H, d.dv), o = view(3, d, d.H, d.dv),
             g = view(4, d, d.H, 1);
  return pdssm_linattn_step(&d, &q, &k, &v, &g, nullptr, d.B, (float*)at(5), &o, nullptr);
}
