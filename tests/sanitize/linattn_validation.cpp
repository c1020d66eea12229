// Host-side validation of the linear-attention calls under AddressSanitizer
// and UndefinedBehaviorSanitizer: workspace queries and refusals on ordinary
// and extreme dims and strides, with launchers that count being reached.
// Pointers are fake device addresses that are never dereferenced.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "pdscan.h"
#include "pdscan_error.h"
#include "pdscan_linattn_launch.h"

static int g_fail = 0, g_launches = 0;
static long long g_grid = 0;

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
hipError_t launch_linattn_form(const LaArgs& a, int, int, hipStream_t) {
  ++g_launches;
  g_grid = (long long)a.segs * a.H * a.slabs * a.njobs;
  if (g_grid > 0x7fffffffll) ++g_fail;
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

static pdssm_linattn_dims dims(int B, int H, int Hk, int L, int dk, int dv, int packed = 0) {
  pdssm_linattn_dims d;
  d.B = B; d.H = H; d.Hk = Hk; d.L = L; d.dk = dk; d.dv = dv;
  d.in_dtype = PDSSM_BF16; d.packed = packed; d.decay_per_head = 0; d.scale = 1.0f;
  return d;
}

static void* at(int slot) { return (void*)(uintptr_t)(0x100000000000ull + ((uint64_t)slot << 42)); }

static pdssm_view view(int slot, const pdssm_linattn_dims& d, int heads, int width) {
  pdssm_view v;
  v.data = at(slot);
  v.stride_t = width;
  v.stride_h = (int64_t)d.L * width;
  v.stride_b = (int64_t)heads * d.L * width;
  return v;
}

int main() {
  size_t n = 0, m = 0;
  const pdssm_linattn_dims shapes[] = {dims(1, 8, 8, 77, 64, 64), dims(4, 8, 8, 4096, 16, 64), dims(16, 24, 24, 2048, 64, 32),
                                       dims(23, 24, 8, 12001, 128, 64, 1), dims(1, 16, 16, 65536, 128, 128), dims(1, 1, 1, 1, 8, 8),
                                       dims(1, 1, 1, 0x7fffff00, 256, 256), dims(1000000, 1, 1, 1, 8, 8), dims(5, 3, 1, 2000000, 256, 8, 1)};
  for (const auto& d : shapes) {
    expect(pdssm_linattn_workspace_bytes(&d, &n), PDSSM_OK, "fwd query");
    expect(pdssm_linattn_bwd_workspace_bytes(&d, &m), PDSSM_OK, "bwd query");
    const int vb = d.packed ? 1 : d.B;
    (void)vb;
    pdssm_view q = view(0, d, d.Hk, d.dk), k = view(1, d, d.Hk, d.dk), v = view(2, d, d.H, d.dv), o = view(3, d, d.H, d.dv);
    pdssm_view g = view(4, d, d.H, 1), gq = view(5, d, d.Hk, d.dk), gk = view(6, d, d.Hk, d.dk), gv = view(7, d, d.H, d.dv), gg = view(8, d, d.H, 1);
    const int32_t* cu = d.packed ? (const int32_t*)at(9) : nullptr;
    float *h0 = (float*)at(10), *hL = (float*)at(11), *ghL = (float*)at(12), *gh0 = (float*)at(13);
    expect(pdssm_linattn_fwd(&d, &q, &k, &v, &g, cu, h0, &o, hL, at(14), n, nullptr), PDSSM_OK, "fwd");
    expect(pdssm_linattn_fwd(&d, &q, &k, &v, &g, cu, h0, &o, hL, at(14), n - 1, nullptr), PDSSM_EWORKSPACE, "fwd short");
    expect(pdssm_linattn_fwd(&d, &q, &k, &v, &g, cu, h0, &v, hL, at(14), n, nullptr), PDSSM_EINVAL, "fwd o = v");
    expect(pdssm_linattn_bwd(&d, &q, &k, &v, &g, cu, h0, &o, ghL, &gq, &gk, &gv, &gg, gh0, at(14), m, nullptr), PDSSM_OK, "bwd");
    expect(pdssm_linattn_bwd(&d, &q, &k, &v, &g, cu, h0, &o, ghL, &gq, &gq, &gv, &gg, gh0, at(14), m, nullptr), PDSSM_EINVAL, "bwd g_k = g_q");
    expect(pdssm_linattn_bwd(&d, &q, &k, &v, &g, cu, h0, &o, ghL, &gq, &gk, &gv, &gg, gh0, at(14), m - 1, nullptr), PDSSM_EWORKSPACE, "bwd short");
  }
  const int reached = g_launches;
  // refused before any launch
  pdssm_linattn_dims d = dims(1, 60000, 60000, 1 << 30, 8, 8);
  expect(pdssm_linattn_workspace_bytes(&d, &n), PDSSM_EUNSUPPORTED, "B*H*L");
  d = dims(1 << 20, 1 << 12, 1, 1, 8, 8);
  expect(pdssm_linattn_workspace_bytes(&d, &n), PDSSM_EUNSUPPORTED, "B*H");
  d = dims(1, 2, 2, 10, 8, 8);
  expect(pdssm_linattn_workspace_bytes(&d, nullptr), PDSSM_EINVAL, "NULL bytes");
  expect(pdssm_linattn_workspace_bytes(nullptr, &n), PDSSM_EINVAL, "NULL dims");
  pdssm_view q = view(0, d, 2, 8), k = view(1, d, 2, 8), v = view(2, d, 2, 8), o = view(3, d, 2, 8), g = view(4, d, 2, 1);
  const int64_t bad[] = {-8, 4, INT64_MIN, INT64_MAX, (int64_t)1 << 62};
  for (int64_t s : bad) {
    pdssm_view w = q;
    w.stride_t = s;
    expect(pdssm_linattn_fwd(&d, &w, &k, &v, &g, nullptr, nullptr, &o, (float*)at(11), at(14), 1 << 20, nullptr), PDSSM_EINVAL, "stride");
    w = o;
    w.stride_h = s;
    expect(pdssm_linattn_fwd(&d, &q, &k, &v, &g, nullptr, nullptr, &w, (float*)at(11), at(14), 1 << 20, nullptr), PDSSM_EINVAL, "o stride");
  }
  // sizes and strides whose product passes 64 bits
  d = dims(1, 1, 1, 0x7fffff00, 8, 8);
  pdssm_linattn_workspace_bytes(&d, &n);
  {
    pdssm_view a = view(0, d, 1, 8), b = view(1, d, 1, 8), c = view(2, d, 1, 8), e = view(3, d, 1, 8), w = view(4, d, 1, 1);
    w.stride_t = (int64_t)1 << 40;
    expect(pdssm_linattn_fwd(&d, &a, &b, &c, &w, nullptr, nullptr, &e, (float*)at(11), at(14), n, nullptr), PDSSM_EINVAL, "long stride");
  }
  d = dims(1, 1 << 20, 1, 1 << 30, 8, 8, 1);
  expect(pdssm_linattn_workspace_bytes(&d, &n), PDSSM_EUNSUPPORTED, "packed H*L");
  d = dims(1, 1 << 20, 1 << 20, 1, 256, 256);
  {
    pdssm_view a = view(0, d, 1 << 20, 256), b = view(1, d, 1 << 20, 256), c = view(2, d, 1 << 20, 256), e = view(3, d, 1 << 20, 256), w = view(4, d, 1 << 20, 1);
    expect(pdssm_linattn_step(&d, &a, &b, &c, &w, (const int32_t*)at(9), 0x7fffffff, (float*)at(11), &e, nullptr), PDSSM_EUNSUPPORTED, "huge pool");
  }
  if (g_launches != reached) ++g_fail;
  // the stride of an axis of one element is not looked at
  d = dims(1, 1, 1, 1, 8, 8);
  pdssm_view odd = q;
  odd.stride_b = -3; odd.stride_h = 5; odd.stride_t = INT64_MIN;
  pdssm_linattn_workspace_bytes(&d, &n);
  expect(pdssm_linattn_fwd(&d, &odd, &k, &v, &g, nullptr, nullptr, &o, (float*)at(11), at(14), n, nullptr), PDSSM_OK, "unit axes");
  // slices of one row-interleaved buffer: told apart, and an overlap of one row found
  d = dims(2, 4, 4, 10, 32, 64);
  const int64_t row = 4 * 128;
  auto slice = [&](int64_t off, int64_t w) {
    pdssm_view x;
    x.data = (char*)at(0) + 2 * off;
    x.stride_b = 10 * row; x.stride_h = w; x.stride_t = row;
    return x;
  };
  pdssm_linattn_bwd_workspace_bytes(&d, &m);
  pdssm_view gq = slice(0, 32), gk = slice(128, 32), gv = slice(256, 64), far = view(5, d, 4, 64), qq = view(6, d, 4, 32);
  g = view(4, d, 4, 1);
  pdssm_view gg = view(8, d, 4, 1);
  pdssm_view vv = view(7, d, 4, 64);
  expect(pdssm_linattn_bwd(&d, &qq, &qq, &vv, &g, nullptr, nullptr, &far, nullptr, &gq, &gk, &gv, &gg, nullptr, at(14), m, nullptr), PDSSM_OK, "slices");
  gv = slice(248, 64);
  expect(pdssm_linattn_bwd(&d, &qq, &qq, &vv, &g, nullptr, nullptr, &far, nullptr, &gq, &gk, &gv, &gg, nullptr, at(14), m, nullptr), PDSSM_EINVAL, "slices that touch");
  gv = slice(264, 64);
  expect(pdssm_linattn_bwd(&d, &qq, &qq, &vv, &g, nullptr, nullptr, &far, nullptr, &gq, &gk, &gv, &gg, nullptr, at(14), m, nullptr), PDSSM_EINVAL, "slices past their row");
  std::printf("ok: %d failures, %d launches\n", g_fail, g_launches);
  return g_fail != 0;
}
