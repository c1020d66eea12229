// Host-side validation of the selective layer's calls under the host
// sanitizers: refusals, workspace queries on ordinary and extreme dims, and
// that what passes fits the device and its workspace.  Pointers are fake device
// addresses that are never dereferenced.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "pdscan.h"
#include "pdscan_error.h"
#include "pdscan_linattn_launch.h"
#include "pdscan_ssm_launch.h"

static int g_fail = 0, g_launches = 0;
static char* g_ws = nullptr;
static size_t g_bytes = 0;

static void fail(const char* what, long long a = 0, long long b = 0) {
  std::fprintf(stderr, "FAIL %s (%lld, %lld)\n", what, a, b);
  ++g_fail;
}

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
// fewer than 2^32 threads along an axis, 65535 rows, every workgroup in 31 bits
static void launch_of(long long blocks, int threads) {
  ++g_launches;
  const LaGrid g = la_grid_rows(blocks, threads);
  if (blocks < 1 || blocks > 0x7fffffffll || (long long)g.x * threads > 0xffffffffll || g.y > 65535) fail("a launch", blocks, threads);
}
// an area of the workspace
static void holds(const void* p, long long bytes) {
  if (!p) return;
  const char* q = (const char*)p;
  if (q < g_ws + kLaHeader || bytes < 0 || q + bytes > g_ws + g_bytes) fail("an area past the workspace", bytes, q - g_ws);
}
static long long units(const SsArgs& a, int per) { return ((long long)a.s.segs * a.G * ss_blocks(a.D / a.G, per) + 7) / 8 * 8; }
static void pieces_ok(const SsArgs& a) {
  if (!a.seg) return;
  // every piece index that a segment of any length can reach
  const long long pieces = a.s.cu ? a.s.L / a.piece + a.s.B : (long long)a.s.B * a.npiece;
  holds(a.seg, pieces * a.D * a.N * 4);
  holds(a.sum, pieces * a.D * 4);
  holds(a.adj, pieces * a.D * a.N * 4);
  if (a.piece < 1 || a.piece % 32) fail("a piece of part of a tile", a.piece);
  if (!a.s.cu && (long long)a.npiece * a.piece < a.s.L) fail("pieces that do not cover", a.npiece, a.piece);
}
static void segs_ok(const SsArgs& a) {
  if (a.s.cu) {
    if (a.s.table) holds(a.s.table, a.s.segs * 16ll);
    if (a.s.segs < (a.s.table ? a.s.L / a.s.seg : 0) + a.s.B) fail("segments of packed sequences", a.s.segs);
  } else if ((long long)a.s.nseg * a.s.seg < a.s.L || (long long)(a.s.nseg - 1) * a.s.seg >= a.s.L || a.s.segs != a.s.nseg * a.s.B) {
    fail("segments that do not cover", a.s.nseg, a.s.seg);
  }
}
hipError_t launch_selscan_fwd(const SsArgs& a, int, hipStream_t) {
  launch_of(units(a, ss_channels(a.N)), 256);
  pieces_ok(a);
  segs_ok(a);
  if (a.seg && !a.s.cu && a.s.nseg > 1 && a.s.seg % a.piece) fail("a run of part of a piece", a.s.seg, a.piece);
  return hipSuccess;
}
hipError_t launch_selscan_state(const SsArgs& a, int, hipStream_t) {
  launch_of(units(a, ss_channels(a.N) * kSsStateGroups), 256);
  pieces_ok(a);
  segs_ok(a);
  return hipSuccess;
}
hipError_t launch_selscan_carry(const SsCarryArgs& a, hipStream_t) {
  launch_of((long long)a.B * (((long long)a.D * a.N + 1023) / 1024), 256);
  return hipSuccess;
}
hipError_t launch_selscan_bwd(const SsArgs& a, int, hipStream_t) {
  const int per = ss_channels(a.N);
  launch_of(units(a, per * kSsBwdGroups), 256 * kSsBwdGroups);
  pieces_ok(a);
  segs_ok(a);
  // tiles: the last one that any piece can name
  const long long t32 = (a.s.L + kSsBwdTile - 1) / kSsBwdTile;
  const long long most = a.s.cu ? (a.seg ? a.s.L / a.piece : 0) + a.s.B - 1 + a.s.L / kSsBwdTile : (long long)a.s.B * t32 - 1;
  holds(a.ckpt, (most + 1) * a.G * ss_blocks(a.D / a.G, per) * ss_shape(a.N).S * 256);
  holds(a.cum, (most + 1) * a.D * 4);
  holds(a.part, 2ll * a.G * ss_blocks(a.D / a.G, per * kSsBwdGroups) * a.rows * a.N * 4);
  holds(a.partA, (long long)a.s.segs * a.D * (a.N + 2) * 4);
  return hipSuccess;
}
static void sum_ok(const SsSumArgs& a) {
  ++g_launches;
  holds(a.part, a.parts * a.width * 4);
  if (a.parts > kSsSumMost) holds(a.mid, kSsSumMid * a.width * 4);
  if ((a.width + 63) / 64 > 0xffffff - 8192) fail("columns of a sum", a.width);
  if (a.share[0] + a.share[1] + a.share[2] < a.width) fail("columns without an output", a.width);
}
hipError_t launch_selscan_fold(const SsFoldArgs& a, int, hipStream_t) { sum_ok(a.sum); return hipSuccess; }
hipError_t launch_ssm_sum(const SsSumArgs& a, hipStream_t) { sum_ok(a); return hipSuccess; }
hipError_t launch_selscan_step(const SsStepArgs& a, int, hipStream_t) {
  const int ns = a.N <= 8 ? 2 : a.N <= 16 ? 4 : a.N <= 32 ? 8 : 16, cw = 256 / ns;
  launch_of((long long)a.B * ((a.D + cw - 1) / cw), 256);
  return hipSuccess;
}
hipError_t launch_conv_fwd(const CvArgs& a, int bf16, hipStream_t) {
  const long long all = cv_units(a, bf16) + (long long)a.B * (a.W - 1) * (a.D / (bf16 ? 8 : 4));
  if (all > 0x7fffffffll) fail("threads past 31 bits", all);
  launch_of((all + 255) / 256, 256);
  return hipSuccess;
}
hipError_t launch_conv_bwd(const CvArgs& a, int, hipStream_t) {
  launch_of((long long)a.parts * ((a.D + 255) / 256), 256);
  holds(a.part, (long long)a.parts * a.D * (a.W + 1) * 4);
  if ((long long)a.parts * kCvBwdStrips < (long long)(a.cu ? 1 : a.B) * a.strips) fail("strips without a part", a.parts, a.strips);
  return hipSuccess;
}
hipError_t launch_conv_step(const CvStepArgs& a, int, hipStream_t) { launch_of((long long)a.B * ((a.D / 4 + 255) / 256), 256); return hipSuccess; }
static void norm_ok(const NmArgs& a, int bf16) {
  launch_of((long long)a.tiles * a.chunks, 256);
  const NmShape n = nm_shape(a.d, bf16);
  if (n.P * n.K * (bf16 ? 8 : 4) < a.d || a.cols % n.P || a.slots * a.cols > 256 || (long long)a.tiles * a.cols < (long long)a.H * n.P)
    fail("rows that are not covered", a.d, a.cols);
  if ((long long)a.chunks * a.slots > 0x7fffffffll || a.rows + (long long)a.chunks * a.slots > 0xffffffffll) fail("rows past 32 bits", a.rows);
}
hipError_t launch_norm_fwd(const NmArgs& a, int bf16, hipStream_t) { norm_ok(a, bf16); return hipSuccess; }
hipError_t launch_norm_bwd(const NmArgs& a, int bf16, hipStream_t) {
  norm_ok(a, bf16);
  holds(a.part, a.chunks * a.part_chunk * 4);
  return hipSuccess;
}
hipError_t launch_linattn_table(const int32_t*, int32_t* table, int32_t* starts, int B, int L, int seg, int segs, hipStream_t) {
  ++g_launches;
  holds(table, segs * 16ll);
  holds(starts, (B + 1) * 4ll);
  if (segs < L / seg + B) fail("a table that is too small", segs);
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

static void* at(int slot) { return (void*)(uintptr_t)(0x10000000000000ull + ((uint64_t)slot << 46)); }
static float* fat(int slot) { return (float*)at(slot); }
static pdssm_view view(int slot, int64_t rows, int64_t heads, int64_t width) {   // [b][t][h][width]
  return pdssm_view{at(slot), rows * heads * width, width, heads * width};
}
static int32_t* cu(int packed) { return packed ? (int32_t*)at(60) : nullptr; }

static int scan_fwd(const pdssm_selscan_dims& d, size_t spare = 0) {
  pdssm_view x = view(1, d.L, 1, d.D), dt = view(2, d.L, 1, d.D), z = view(3, d.L, 1, d.D), y = view(4, d.L, 1, d.D);
  pdssm_view b = view(5, d.L, d.G, d.N), c = view(6, d.L, d.G, d.N);
  size_t n = 0;
  int rc = pdssm_selscan_workspace_bytes(&d, &n);
  if (rc) return rc;
  g_ws = (char*)at(50);
  g_bytes = n;
  return pdssm_selscan_fwd(&d, &x, &dt, fat(7), &b, &c, fat(8), &z, fat(9), cu(d.packed), fat(10), &y, fat(11), n ? g_ws : nullptr, n - spare, nullptr);
}
static int scan_bwd(const pdssm_selscan_dims& d, size_t spare = 0) {
  pdssm_view x = view(1, d.L, 1, d.D), dt = view(2, d.L, 1, d.D), z = view(3, d.L, 1, d.D), gy = view(4, d.L, 1, d.D);
  pdssm_view b = view(5, d.L, d.G, d.N), c = view(6, d.L, d.G, d.N), gb = view(12, d.L, d.G, d.N), gc = view(13, d.L, d.G, d.N);
  pdssm_view gx = view(14, d.L, 1, d.D), gd = view(15, d.L, 1, d.D), gz = view(16, d.L, 1, d.D);
  size_t n = 0;
  int rc = pdssm_selscan_bwd_workspace_bytes(&d, &n);
  if (rc) return rc;
  g_ws = (char*)at(50);
  g_bytes = n;
  return pdssm_selscan_bwd(&d, &x, &dt, fat(7), &b, &c, fat(8), &z, fat(9), cu(d.packed), fat(10), &gy, fat(11), &gx, &gd, fat(17), &gb, &gc,
                           fat(18), &gz, fat(19), fat(20), g_ws, n - spare, nullptr);
}
static int scan_step(pdssm_selscan_dims d, int slots) {
  d.L = 1;
  d.packed = 0;
  pdssm_view x = view(1, 1, 1, d.D), dt = view(2, 1, 1, d.D), y = view(4, 1, 1, d.D), b = view(5, 1, d.G, d.N), c = view(6, 1, d.G, d.N);
  return pdssm_selscan_step(&d, &x, &dt, fat(7), &b, &c, nullptr, nullptr, nullptr, (int32_t*)at(60), slots, fat(10), &y, nullptr);
}
static int conv_both(const pdssm_conv_dims& d) {
  pdssm_view x = view(1, d.L, 1, d.D), y = view(2, d.L, 1, d.D), gx = view(3, d.L, 1, d.D);
  int rc = pdssm_conv_fwd(&d, &x, fat(4), fat(5), cu(d.packed), at(6), &y, at(7), nullptr);
  size_t n = 0;
  const int rq = pdssm_conv_bwd_workspace_bytes(&d, &n);
  if (rq != rc) fail("query and call differ", rq, rc);
  if (rc) return rc;
  g_ws = (char*)at(50);
  g_bytes = n;
  return pdssm_conv_bwd(&d, &x, fat(4), fat(5), cu(d.packed), at(6), &y, at(8), &gx, fat(9), fat(10), at(11), g_ws, n, nullptr);
}
static int norm_both(const pdssm_norm_dims& d, bool near) {
  pdssm_view v[6];
  for (int i = 0; i < 6; ++i) {
    v[i] = view(1 + i, d.L, d.H, d.d);
    if (!near) v[i].stride_h = (int64_t)d.L * d.d, v[i].stride_t = d.d;
  }
  const bool gate = d.gate != PDSSM_GATE_NONE;
  int rc = pdssm_norm_fwd(&d, &v[0], fat(10), gate ? &v[1] : nullptr, &v[2], fat(11), &v[3], nullptr);
  size_t n = 0;
  const int rq = pdssm_norm_bwd_workspace_bytes(&d, &n);
  if (rc) return rc;
  if (rq) return rq;
  g_ws = (char*)at(50);
  g_bytes = n;
  return pdssm_norm_bwd(&d, &v[0], fat(10), gate ? &v[1] : nullptr, fat(11), &v[2], &v[3], fat(12), gate ? &v[4] : nullptr, fat(13), g_ws, n, nullptr);
}

int main() {
  const pdssm_selscan_dims s = {2, 700, 64, 16, 2, PDSSM_BF16, 0, 1};
  const pdssm_conv_dims c = {2, 70, 64, 4, PDSSM_BF16, 0, 1};
  const pdssm_norm_dims m = {2, 3, 7, 64, PDSSM_BF16, PDSSM_GATE_AFTER, 1, 1e-5f};
  expect(scan_fwd(s), PDSSM_OK, "scan");
  expect(scan_bwd(s), PDSSM_OK, "scan gradient");
  expect(scan_step(s, 5), PDSSM_OK, "scan step");
  expect(conv_both(c), PDSSM_OK, "conv");
  expect(norm_both(m, true), PDSSM_OK, "norm");
  // refusals reach no launch
  const int before = g_launches;
  auto S = [&](auto set, int want, const char* what) {
    pdssm_selscan_dims d = s;
    set(d);
    expect(scan_fwd(d), want, what);
    expect(scan_bwd(d), want, what);
  };
  S([](auto& d) { d.B = 0; }, PDSSM_EINVAL, "no sequences");
  S([](auto& d) { d.L = -1; }, PDSSM_EINVAL, "negative steps");
  S([](auto& d) { d.N = 0; }, PDSSM_EINVAL, "no states");
  S([](auto& d) { d.G = 3; }, PDSSM_EINVAL, "groups that do not divide");
  S([](auto& d) { d.G = 16; }, PDSSM_EUNSUPPORTED, "groups of four channels");
  S([](auto& d) { d.N = 12; }, PDSSM_EUNSUPPORTED, "twelve states");
  S([](auto& d) { d.N = 72; }, PDSSM_EUNSUPPORTED, "72 states");
  S([](auto& d) { d.D = 60; }, PDSSM_EUNSUPPORTED, "60 channels");
  S([](auto& d) { d.D = 1 << 21; }, PDSSM_EUNSUPPORTED, "too many channels");
  S([](auto& d) { d.in_dtype = 2; }, PDSSM_EINVAL, "type");
  S([](auto& d) { d.packed = 2; }, PDSSM_EINVAL, "packed");
  S([](auto& d) { d.softplus = -1; }, PDSSM_EINVAL, "softplus");
  S([](auto& d) { d.B = d.L = 0x7fffffff; }, PDSSM_EUNSUPPORTED, "rows past 31 bits");
  S([](auto& d) { d.B = 0x7fffff00; d.L = 1; d.D = 1 << 20; }, PDSSM_EUNSUPPORTED, "workgroups past 31 bits");
  expect(scan_fwd(s, 1), PDSSM_EWORKSPACE, "short workspace");
  expect(scan_bwd(s, 1), PDSSM_EWORKSPACE, "short workspace");
  expect(scan_step(s, 0), PDSSM_EINVAL, "no slots");
  size_t n;
  expect(pdssm_selscan_workspace_bytes(nullptr, &n), PDSSM_EINVAL, "no dims");
  expect(pdssm_selscan_workspace_bytes(&s, nullptr), PDSSM_EINVAL, "no answer");
  {
    pdssm_view x = view(1, 700, 1, 64), b = view(5, 700, 2, 16), y = view(4, 700, 1, 64);
    size_t need = 0;
    pdssm_selscan_workspace_bytes(&s, &need);
    auto call = [&](pdssm_view* xx, pdssm_view* yy, const int32_t* k, const float* A, void* ws) {
      return pdssm_selscan_fwd(&s, xx, &x, A, &b, &b, nullptr, nullptr, nullptr, k, nullptr, yy, fat(11), ws, need, nullptr);
    };
    pdssm_view odd = x, half = x, zero = y, neg = x;
    odd.data = (char*)odd.data + 2;
    half.stride_t = 68;
    zero.stride_t = 0;
    neg.stride_b = -64;
    expect(call(nullptr, &y, nullptr, fat(7), at(50)), PDSSM_EINVAL, "no x");
    expect(call(&odd, &y, nullptr, fat(7), at(50)), PDSSM_EINVAL, "misaligned x");
    expect(call(&half, &y, nullptr, fat(7), at(50)), PDSSM_EINVAL, "odd stride");
    expect(call(&neg, &y, nullptr, fat(7), at(50)), PDSSM_EINVAL, "negative stride");
    expect(call(&x, &zero, nullptr, fat(7), at(50)), PDSSM_EINVAL, "rows of y overlap");
    expect(call(&x, &x, nullptr, fat(7), at(50)), PDSSM_EINVAL, "y is x");
    expect(call(&x, &y, (int32_t*)at(60), fat(7), at(50)), PDSSM_EINVAL, "offsets without packed");
    expect(call(&x, &y, nullptr, nullptr, at(50)), PDSSM_EINVAL, "no A");
    expect(call(&x, &y, nullptr, fat(7), nullptr), PDSSM_EINVAL, "no workspace");
    expect(call(&x, &y, nullptr, fat(7), at(4)), PDSSM_EINVAL, "workspace is y");
  }
  auto C = [&](auto set, int want, const char* what) {
    pdssm_conv_dims d = c;
    set(d);
    expect(conv_both(d), want, what);
  };
  C([](auto& d) { d.W = 1; }, PDSSM_EUNSUPPORTED, "one tap");
  C([](auto& d) { d.W = 5; }, PDSSM_EUNSUPPORTED, "five taps");
  C([](auto& d) { d.silu = 2; }, PDSSM_EINVAL, "silu");
  C([](auto& d) { d.D = 12; }, PDSSM_EUNSUPPORTED, "twelve channels");
  C([](auto& d) { d.L = 0x7fffff00; d.B = 1; }, PDSSM_EUNSUPPORTED, "threads past 31 bits");
  auto M = [&](auto set, int want, const char* what) {
    pdssm_norm_dims d = m;
    set(d);
    expect(norm_both(d, true), want, what);
  };
  M([](auto& d) { d.eps = 0; }, PDSSM_EINVAL, "eps");
  M([](auto& d) { d.eps = 1e-40f; }, PDSSM_EINVAL, "eps below the normal numbers");
  M([](auto& d) { d.gate = 3; }, PDSSM_EINVAL, "gate");
  M([](auto& d) { d.d = 12; }, PDSSM_EUNSUPPORTED, "rows of twelve");
  M([](auto& d) { d.d = 8200; }, PDSSM_EUNSUPPORTED, "long rows");
  M([](auto& d) { d.B = 1 << 30; d.L = 8; }, PDSSM_EUNSUPPORTED, "rows past 31 bits");
  M([](auto& d) { d.B = d.L = 1; d.H = 1 << 16; d.d = 8192; }, PDSSM_EUNSUPPORTED, "weights whose sums pass a launch");
  if (g_launches != before) fail("a refused call launched", g_launches - before);

  // every size that passes covers its rows and stays inside its workspace
  long long calls = 0;
  for (int B : {1, 2, 3, 7, 40, 300, 70000})
    for (int L : {1, 31, 64, 129, 300, 513, 1000, 4097, 65536, 1000003})
      for (int D : {8, 24, 96, 768, 4096, 1 << 20})
        for (int N : {8, 16, 24, 64})
          for (int G : {1, 3})
            for (int packed = 0; packed < 2; ++packed) {
              if (D % (8 * G)) continue;
              const pdssm_selscan_dims d = {B, L, D, N, G, PDSSM_F32, packed, 1};
              const int l0 = g_launches;
              int rc = scan_fwd(d);
              if (rc && g_launches != l0) fail("a refused call launched", B, L);
              const int l1 = g_launches;
              rc = scan_bwd(d);
              if (rc && g_launches != l1) fail("a refused call launched", B, L);
              calls += 2;
              if (N == 8 && G == 1) {
                for (int W = 2; W <= 4; ++W) {
                  const pdssm_conv_dims e = {B, L, D, W, W & 1, packed, 1};
                  conv_both(e);
                  ++calls;
                }
              }
            }
  for (int B : {1, 3, 1000})
    for (int H : {1, 2, 5, 24, 700})
      for (int L : {1, 7, 2048, 1000000})
        for (int d = 8; d <= 8192; d += d < 128 ? 8 : d < 1024 ? 72 : 1024)
          for (int f = 0; f < 8; ++f) {
            const pdssm_norm_dims e = {B, H, L, d, f & 1, f >> 1 & 1 ? PDSSM_GATE_AFTER : PDSSM_GATE_NONE, f >> 2 & 1, 1e-5f};
            norm_both(e, f & 2);
            ++calls;
          }
  // pieces and tiles of packed sequences of any offsets, as the tables' kernel cuts them
  unsigned seed = 1;
  auto rnd = [&](int n) { seed = seed * 1664525u + 1013904223u; return (int)((seed >> 8) % (unsigned)n); };
  for (int turn = 0; turn < 3000; ++turn) {
    const int B = 1 + rnd(6), L = 1 + rnd(3000), D = 8 * (1 + rnd(40));
    const pdscan::SsSplit p = pdscan::ss_split(B, L, 1, (D + 15) / 16, 3, (D + 63) / 64, true);
    int off[8];
    for (int i = 0; i <= B; ++i) off[i] = turn % 3 ? rnd(L + 1) : rnd(3 * L) - L;
    if (turn % 4 == 0)
      for (int i = 1; i <= B; ++i) off[i] = off[i] < off[i - 1] ? off[i - 1] : off[i];
    struct Row { int b, t0, len; };
    auto table = [&](int seg, int most, int* first, std::vector<Row>& rows) {
      for (int b = 0; b < B; ++b) {
        int t0 = off[b], t1 = off[b + 1];
        t0 = t0 < 0 ? 0 : t0 > L ? L : t0;
        t1 = t1 < t0 ? t0 : t1 > L ? L : t1;
        first[b] = (int)rows.size() < most ? (int)rows.size() : most;
        const int len = t1 - t0, n = len <= seg ? 1 : (len - 1) / seg + 1;
        for (int i = 0; i < n && (int)rows.size() < most; ++i) rows.push_back({b, t0 + i * seg, len - i * seg < seg ? len - i * seg : seg});
      }
    };
    int pieces[8], runs[8];
    std::vector<Row> pr, rr;
    if (p.states) table(p.piece, p.pieces, pieces, pr);
    table(p.cut ? p.seg : L, p.segs, runs, rr);
    const long long tiles = p.pieces + (L + 31) / 32;
    std::vector<int> owner(tiles, -1);
    for (int sid = 0; sid < (int)pr.size(); ++sid)   // the state pass writes them
      for (int t = 0; t < pr[sid].len; t += 32) {
        const long long at = pdscan::ss_tile_of(0, pr[sid].b, sid, pr[sid].t0, t, 32);
        if (at < 0 || at >= tiles) fail("a tile past the workspace", at, tiles);
        else if (turn % 4 == 0 && owner[at] >= 0) fail("two tiles in one place", at);
        else owner[at] = sid;
      }
    for (int sid = 0; sid < (int)rr.size(); ++sid)   // the gradient reads them
      for (int t = 0; t < rr[sid].len; t += 32) {
        const int pc = p.states ? t / p.piece : 0;
        const int piece = p.states ? pdscan::ss_piece_at(pdscan::ss_piece_at(pieces[rr[sid].b], p.cut ? (sid - runs[rr[sid].b]) * p.run : 0, p.pieces), pc, p.pieces) : rr[sid].b;
        if (piece < 0 || piece >= p.pieces) fail("a piece past the workspace", piece, p.pieces);
        const long long at = pdscan::ss_tile_of(0, rr[sid].b, piece, rr[sid].t0 + (p.states ? pc * p.piece : 0), p.states ? t - pc * p.piece : t, 32);
        if (at < 0 || at >= tiles) fail("a tile past the workspace", at, tiles);
        if (turn % 4 == 0 && p.states && (at < 0 || at >= tiles || owner[at] != piece)) fail("a tile that nobody wrote", at);
      }
  }
  std::printf("ok: %d failures, %lld calls, %d launches\n", g_fail, calls, g_launches);
  return g_fail != 0;
}
