// C ABI of the selective scan, the short convolution and the norm
// (pdssm_selscan_*, pdssm_conv_*, pdssm_norm_*): argument validation (host
// only, before any HIP call), workspace layout and the order of the launches.
// The contract of every entry point is in include/pdscan.h.

#include <hip/hip_runtime_api.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "pdscan.h"
#include "pdscan_args.h"
#include "pdscan_error.h"
#include "pdscan_linattn_launch.h"
#include "pdscan_ssm_launch.h"
#include "pdscan_ssm_plan.h"

namespace {

using pdscan::CvArgs;
using pdscan::LaView;
using pdscan::NmArgs;
using pdscan::Span;
using pdscan::SsArgs;
using pdscan::SsSplit;
using pdscan::SsSumArgs;
using pdscan::check_overlap;
using pdscan::dense;
using pdscan::dense_ok;
using pdscan::launched;
using pdscan::set_error;
using pdscan::view_span;

constexpr int64_t kMost = 0x7fffff00;  // rows, workgroups and threads are numbered in 31 bits

// Arguments of a call as they are checked: first each by itself, then what may not overlap.
struct Args {
  Span in[12], out[12];
  int nin = 0, nout = 0, rc = PDSSM_OK;
  int es, D;
  int64_t B, L;                        // rows of the batch axis, steps

  void view(bool output, LaView& v, const char* name, const pdssm_view* a, bool required, int64_t heads, int width) {
    v = LaView{};
    if (rc || (!a && !required)) return;
    const int64_t ext[3] = {B, heads, L};
    Span s;
    rc = view_span(s, v, name, a, ext, width, es);
    if (!rc) add(output, s);
  }
  // [B,L,D] without a head axis
  void rows(bool output, LaView& v, const char* name, const pdssm_view* a, bool required = true) {
    view(output, v, name, a, required, 1, D);
  }
  void flat(bool output, const char* name, const void* p, size_t bytes, bool required, uintptr_t align = 16) {
    if (rc) return;
    const Span s = dense(name, p, bytes);
    rc = dense_ok(s, required, align);
    if (!rc && p) add(output, s);
  }
  void add(bool output, const Span& s) {
    if (output) out[nout++] = s;
    else in[nin++] = s;
  }
  int check(void* workspace = nullptr, size_t have = 0, size_t need = 0) {
    if (rc) return rc;
    if (need || (workspace && have)) {
      flat(true, "workspace", workspace, need ? need : have, true);
      if (rc) return rc;
      if (have < need) return set_error(PDSSM_EWORKSPACE, "workspace of %zu bytes < %zu needed", have, need);
    }
    return check_overlap(in, nin, out, nout);
  }
};

int check_rows(int B, int L, int D, int in_dtype, int packed, bool step) {
  if (B < 1 || L < 1 || D < 1) return set_error(PDSSM_EINVAL, "dims must be >= 1 (B=%d L=%d D=%d)", B, L, D);
  if (in_dtype != PDSSM_F32 && in_dtype != PDSSM_BF16)
    return set_error(PDSSM_EINVAL, "in_dtype must be PDSSM_F32 or PDSSM_BF16 (got %d)", in_dtype);
  if (packed != 0 && packed != 1) return set_error(PDSSM_EINVAL, "packed must be 0 or 1 (got %d)", packed);
  if (step && (L != 1 || packed)) return set_error(PDSSM_EINVAL, "a step has L=1 and packed=0 (got L=%d packed=%d)", L, packed);
  if (D % 8 || D > pdscan::kSsMaxD)
    return set_error(PDSSM_EUNSUPPORTED, "D=%d must be a multiple of 8, at most %d", D, pdscan::kSsMaxD);
  if (L > kMost || (int64_t)(packed ? 1 : B) * L > kMost || B > kMost)
    return set_error(PDSSM_EUNSUPPORTED, "B=%d sequences of L=%d steps are too many", B, L);
  return PDSSM_OK;
}

struct Layout {
  size_t at = pdscan::kLaHeader;
  size_t put(size_t bytes) {
    const size_t here = at;
    at += pdscan::la_align(bytes);
    return here;
  }
};

int check_packed(int packed, const int32_t* cu) {
  return !packed && cu ? set_error(PDSSM_EINVAL, "cu_seqlens given with packed = 0") : PDSSM_OK;
}

// ---- convolution

int check_conv(const pdssm_conv_dims* d, bool step) {
  if (!d) return set_error(PDSSM_EINVAL, "dims is NULL");
  int rc = check_rows(d->B, d->L, d->D, d->in_dtype, d->packed, step);
  if (rc) return rc;
  if (d->silu != 0 && d->silu != 1) return set_error(PDSSM_EINVAL, "silu must be 0 or 1 (got %d)", d->silu);
  if (d->W < pdscan::kCvMinW || d->W > pdscan::kCvMaxW)
    return set_error(PDSSM_EUNSUPPORTED, "W=%d must be %d to %d", d->W, pdscan::kCvMinW, pdscan::kCvMaxW);
  // threads of the largest launches: strips of rows, and the states' vectors of four
  const int64_t strips = (int64_t)(d->packed ? 1 : d->B) * ((d->L + pdscan::kCvRows - 1) / pdscan::kCvRows);
  if (strips * (d->D / 4) > kMost || (int64_t)d->B * (d->W - 1) * (d->D / 4) + strips * (d->D / 4) > kMost)
    return set_error(PDSSM_EUNSUPPORTED, "B=%d sequences of L=%d steps and D=%d channels are too many", d->B, d->L, d->D);
  return PDSSM_OK;
}

struct CvWs {
  int strips, parts;
  int64_t width;
  size_t part, mid, total;
};
CvWs conv_ws(const pdssm_conv_dims* d) {
  CvWs w;
  w.strips = (d->L + pdscan::kCvBwdRows - 1) / pdscan::kCvBwdRows;
  const int64_t all = (int64_t)(d->packed ? 1 : d->B) * w.strips;
  w.parts = (int)((all + pdscan::kCvBwdStrips - 1) / pdscan::kCvBwdStrips);
  w.width = (int64_t)d->D * (d->W + 1);
  Layout l;
  w.part = l.put((size_t)w.parts * w.width * 4);
  w.mid = l.put(w.parts > pdscan::kSsSumMost ? (size_t)pdscan::kSsSumMid * w.width * 4 : 0);
  w.total = l.at;
  return w;
}

// ---- scan

int check_scan(const pdssm_selscan_dims* d, bool step) {
  if (!d) return set_error(PDSSM_EINVAL, "dims is NULL");
  int rc = check_rows(d->B, d->L, d->D, d->in_dtype, d->packed, step);
  if (rc) return rc;
  if (d->N < 1 || d->G < 1) return set_error(PDSSM_EINVAL, "dims must be >= 1 (N=%d G=%d)", d->N, d->G);
  if (d->softplus != 0 && d->softplus != 1) return set_error(PDSSM_EINVAL, "softplus must be 0 or 1 (got %d)", d->softplus);
  if (d->D % d->G) return set_error(PDSSM_EINVAL, "D=%d is not a multiple of G=%d", d->D, d->G);
  if (d->N % 8 || d->N > pdscan::kSsMaxN)
    return set_error(PDSSM_EUNSUPPORTED, "N=%d must be a multiple of 8, at most %d", d->N, pdscan::kSsMaxN);
  if (d->D / d->G % 8) return set_error(PDSSM_EUNSUPPORTED, "D / G = %d must be a multiple of 8", d->D / d->G);
  return PDSSM_OK;
}

// Workgroups of the widest launch over so many segments: channel blocks of the fewest channels.
int scan_grid(const pdssm_selscan_dims* d, const SsSplit& s) {
  const int64_t blocks = (int64_t)d->G * pdscan::ss_blocks(d->D / d->G, pdscan::ss_channels(d->N));
  if (s.pieces * blocks > kMost / 2 || (int64_t)d->B * (((int64_t)d->D * d->N + 1023) / 1024) > kMost)
    return set_error(PDSSM_EUNSUPPORTED, "too many pieces and channels (%d, %d)", s.pieces, d->D);
  return PDSSM_OK;
}

struct ScanWs {
  SsSplit split;
  size_t table, pieces, run_table, runs, seg, adj, sum, ckpt, cum, part, partA, mid, total;
  int blocks;                          // (gradient) channel blocks of a group
};

// Tables of packed sequences, contributions of pieces and their sums.
void put_pieces(ScanWs& w, Layout& l, const pdssm_selscan_dims* d, bool bwd) {
  const SsSplit& p = w.split;
  const size_t state = (size_t)p.pieces * d->D * d->N * 4;
  w.table = w.pieces = w.run_table = w.runs = w.seg = w.adj = w.sum = l.at;
  if (!p.states) return;
  if (d->packed) {
    w.table = l.put((size_t)p.pieces * 16);
    w.pieces = l.put(((size_t)d->B + 1) * 4);
    if (p.cut) {
      w.run_table = l.put((size_t)p.segs * 16);
      w.runs = l.put(((size_t)d->B + 1) * 4);
    }
  }
  w.seg = l.put(state);
  if (bwd && p.cut) w.adj = l.put(state);
  w.sum = l.put((size_t)p.pieces * d->D * 4);
}

int64_t scan_blocks(const pdssm_selscan_dims* d, int groups) {
  return (int64_t)d->G * pdscan::ss_blocks(d->D / d->G, pdscan::ss_channels(d->N) * groups);
}

// Workgroups of four waves that a compute unit holds, by their registers.
int per_cu(const pdssm_selscan_dims* d) { return pdscan::ss_shape(d->N).S >= 8 ? 2 : 3; }

ScanWs scan_ws(const pdssm_selscan_dims* d) {
  ScanWs w = {};
  w.split = pdscan::ss_split(d->B, d->L, d->packed, scan_blocks(d, 1), per_cu(d), scan_blocks(d, pdscan::kSsStateGroups), false);
  Layout l;
  put_pieces(w, l, d, false);
  w.total = w.split.states ? l.at : 0;
  return w;
}

ScanWs scan_bwd_ws(const pdssm_selscan_dims* d) {
  ScanWs w = {};
  const int per = pdscan::ss_channels(d->N);
  const size_t rows = (size_t)(d->packed ? 1 : d->B) * d->L;
  w.blocks = pdscan::ss_blocks(d->D / d->G, per * pdscan::kSsBwdGroups);
  w.split = pdscan::ss_split(d->B, d->L, d->packed, scan_blocks(d, pdscan::kSsBwdGroups), per_cu(d),
                             scan_blocks(d, pdscan::kSsStateGroups), true);
  Layout l;
  put_pieces(w, l, d, true);
  const size_t perseq = ((size_t)d->L + pdscan::kSsBwdTile - 1) / pdscan::kSsBwdTile;
  const size_t tiles = d->packed ? (size_t)w.split.pieces + perseq : d->B * perseq;
  const pdscan::SsShape shape = pdscan::ss_shape(d->N);
  w.ckpt = l.put(tiles * scan_blocks(d, 1) * shape.S * 64 * 4);
  w.cum = l.put(tiles * d->D * 4);
  w.part = l.put(2 * (size_t)d->G * w.blocks * rows * d->N * 4);
  w.partA = l.put((size_t)w.split.segs * d->D * (d->N + 2) * 4);
  w.mid = l.put(w.split.segs > pdscan::kSsSumMost ? (size_t)pdscan::kSsSumMid * d->D * (d->N + 2) * 4 : 0);
  w.total = l.at;
  return w;
}

// The arguments that every pass of the scan reads.
struct ScanIn {
  const pdssm_view *x, *dt, *Bm, *Cm, *z;
  const float *A, *skip, *bias;
};
void scan_in(Args& c, SsArgs& a, const pdssm_selscan_dims* d, const ScanIn& i) {
  c.es = d->in_dtype == PDSSM_BF16 ? 2 : 4;
  c.B = d->packed ? 1 : d->B;
  c.L = d->L;
  c.D = d->D;
  c.rows(false, a.x, "x", i.x);
  c.rows(false, a.dt, "dt", i.dt);
  c.flat(false, "A", i.A, (size_t)d->D * d->N * 4, true);
  c.view(false, a.Bm, "Bm", i.Bm, true, d->G, d->N);
  c.view(false, a.Cm, "Cm", i.Cm, true, d->G, d->N);
  c.flat(false, "skip", i.skip, (size_t)d->D * 4, false);
  c.rows(false, a.z, "z", i.z, false);
  c.flat(false, "dt_bias", i.bias, (size_t)d->D * 4, false);
  a.A = i.A; a.skip = i.skip; a.bias = i.bias;
  a.D = d->D; a.N = d->N; a.G = d->G; a.softplus = d->softplus;
  a.rows = c.B * c.L;
}

// The launches before a scan's last: tables, states at the pieces' starts (and,
// for a gradient, at the tiles'), the adjoint's at the runs' ends.  Leaves in
// `a` what the last one reads.
hipError_t scan_states(SsArgs& a, const pdssm_selscan_dims* d, const ScanWs& w, const int32_t* cu, unsigned char* ws,
                       size_t bytes, bool bwd, hipStream_t st) {
  const SsSplit& p = w.split;
  const int bf16 = d->in_dtype == PDSSM_BF16;
  a.header = ws && bytes >= pdscan::kLaHeader ? (uint32_t*)ws : nullptr;
  a.piece = p.piece; a.npiece = p.npiece; a.run = p.run; a.npieces = p.pieces;
  pdscan::SsSegs pieces = {cu, nullptr, d->B, d->L, p.npiece, p.piece, p.pieces};
  pdscan::SsSegs runs = {cu, nullptr, d->B, d->L, p.nseg, p.seg, p.segs};
  hipError_t e = hipSuccess;
  if (p.states) {
    a.seg = (float*)(ws + w.seg);
    a.sum = (float*)(ws + w.sum);
    if (bwd && p.cut) a.adj = (float*)(ws + w.adj);
    if (cu) {
      pieces.table = (const int32_t*)(ws + w.table);
      a.pieces = (const int32_t*)(ws + w.pieces);
      e = pdscan::launch_linattn_table(cu, (int32_t*)(ws + w.table), (int32_t*)(ws + w.pieces), d->B, d->L, p.piece, p.pieces, st);
      if (p.cut) {
        runs.table = (const int32_t*)(ws + w.run_table);
        a.runs = (const int32_t*)(ws + w.runs);
        if (e == hipSuccess)
          e = pdscan::launch_linattn_table(cu, (int32_t*)(ws + w.run_table), (int32_t*)(ws + w.runs), d->B, d->L, p.seg, p.segs, st);
      }
    }
  }
  if (p.states || bwd) {
    a.s = pieces;
    if (e == hipSuccess) e = pdscan::launch_selscan_state(a, bf16, st);
  }
  if (p.states) {
    pdscan::SsCarryArgs c = {};
    c.A = a.A;
    c.user[0] = a.h0;
    c.user[1] = a.ghL;
    c.seg[0] = a.seg;
    c.seg[1] = a.adj;
    c.sum = a.sum;
    c.starts = a.pieces;
    c.B = d->B; c.D = d->D; c.N = d->N; c.npiece = p.npiece;
    if (e == hipSuccess) e = pdscan::launch_selscan_carry(c, st);
  }
  a.s = runs;
  return e;
}

// ---- norm

int check_norm(const pdssm_norm_dims* d) {
  if (!d) return set_error(PDSSM_EINVAL, "dims is NULL");
  if (d->B < 1 || d->H < 1 || d->L < 1 || d->d < 1)
    return set_error(PDSSM_EINVAL, "dims must be >= 1 (B=%d H=%d L=%d d=%d)", d->B, d->H, d->L, d->d);
  if (d->in_dtype != PDSSM_F32 && d->in_dtype != PDSSM_BF16)
    return set_error(PDSSM_EINVAL, "in_dtype must be PDSSM_F32 or PDSSM_BF16 (got %d)", d->in_dtype);
  if (d->gate < PDSSM_GATE_NONE || d->gate > PDSSM_GATE_AFTER)
    return set_error(PDSSM_EINVAL, "gate must be a pdssm_gate (got %d)", d->gate);
  if (d->per_head != 0 && d->per_head != 1) return set_error(PDSSM_EINVAL, "per_head must be 0 or 1 (got %d)", d->per_head);
  if (!(d->eps >= FLT_MIN) || !std::isfinite(d->eps)) return set_error(PDSSM_EINVAL, "eps must be > 0, a normal number");
  if (d->d % 8 || d->d > pdscan::kNmMaxD)
    return set_error(PDSSM_EUNSUPPORTED, "d=%d must be a multiple of 8, at most %d", d->d, pdscan::kNmMaxD);
  if ((int64_t)d->B * d->L > kMost / 2 || (int64_t)d->H * 256 > kMost || d->L > kMost / 2)
    return set_error(PDSSM_EUNSUPPORTED, "B=%d sequences of L=%d rows and H=%d heads are too many", d->B, d->L, d->H);
  // a gradient's last sum takes four threads a column, w's and res_scale's, and a launch fewer than 2^32
  if (d->per_head && (int64_t)d->H * d->d >= 1 << 29)
    return set_error(PDSSM_EUNSUPPORTED, "weights of H=%d heads of d=%d elements are too many", d->H, d->d);
  return PDSSM_OK;
}

bool norm_near(const pdssm_norm_dims* d, const pdssm_view* x) { return d->H > 1 && x && x->stride_h < x->stride_t; }

// Workgroups along the rows of a gradient: enough to fill the card, few enough that their sums are small.
constexpr int kNormChunks = 1024;
int norm_most(const pdssm_norm_dims* d) {
  const int64_t tiles = ((int64_t)d->H * pdscan::nm_shape(d->d, d->in_dtype == PDSSM_BF16).P + 255) / 256;
  return tiles >= kNormChunks ? 1 : (int)(kNormChunks / tiles);
}

struct NormWs {
  size_t part, mid, total;
};
NormWs norm_ws(const pdssm_norm_dims* d) {   // (room for the sums of res_scale in any case)
  NormWs n;
  const int64_t most = norm_most(d), sums = d->per_head ? most : most * d->H;   // parts of the last sum
  Layout l;
  n.part = l.put((size_t)most * d->H * d->d * 8);
  n.mid = l.put(sums > pdscan::kSsSumMost ? (size_t)pdscan::kSsSumMid * (d->per_head ? d->H : 1) * d->d * 8 : 0);
  n.total = l.at;
  return n;
}

void norm_in(Args& c, NmArgs& a, const pdssm_norm_dims* d, const pdssm_view* x, const float* w, const pdssm_view* z,
             const float* s) {
  c.es = d->in_dtype == PDSSM_BF16 ? 2 : 4;
  c.B = d->B;
  c.L = d->L;
  const size_t wide = (size_t)(d->per_head ? d->H : 1) * d->d * 4;
  c.view(false, a.x, "x", x, true, d->H, d->d);
  c.flat(false, "w", w, wide, true);
  if (!c.rc && d->gate == PDSSM_GATE_NONE && z) c.rc = set_error(PDSSM_EINVAL, "z given without a gate");
  c.view(false, a.z, "z", z, d->gate != PDSSM_GATE_NONE, d->H, d->d);
  c.flat(false, "res_scale", s, wide, false);
  a.w = w; a.s = s;
  a.B = d->B; a.H = d->H; a.L = d->L; a.d = d->d; a.gate = d->gate; a.per_head = d->per_head;
  a.eps = d->eps;
  a.rows = (long long)d->B * d->L;
}

template <typename W>
int answer(size_t* bytes, const W& w) {
  if (!bytes) return set_error(PDSSM_EINVAL, "bytes is NULL");
  *bytes = w.total;
  pdscan::clear_error();
  return PDSSM_OK;
}

int check_slots(int B, const int32_t* idx, int32_t n_slots, int64_t state) {
  if (n_slots < 1) return set_error(PDSSM_EINVAL, "n_slots must be >= 1 (got %d)", n_slots);
  if (!idx && n_slots < B) return set_error(PDSSM_EINVAL, "n_slots=%d < B=%d without state_idx", n_slots, B);
  if (n_slots > (1ll << 50) / state) return set_error(PDSSM_EUNSUPPORTED, "n_slots=%d is too large", n_slots);
  return PDSSM_OK;
}

}  // namespace

extern "C" {

int pdssm_conv_fwd(const pdssm_conv_dims* dims, const pdssm_view* x, const float* w, const float* bias,
                   const int32_t* cu_seqlens, const void* x0, const pdssm_view* y, void* x_L, void* stream) {
  int rc = check_conv(dims, false);
  if (rc || (rc = check_packed(dims->packed, cu_seqlens))) return rc;
  const pdssm_conv_dims& d = *dims;
  CvArgs a = {};
  Args c;
  c.es = d.in_dtype == PDSSM_BF16 ? 2 : 4;
  c.B = d.packed ? 1 : d.B; c.L = d.L; c.D = d.D;
  const size_t state = (size_t)d.B * (d.W - 1) * d.D * c.es;
  c.rows(false, a.x, "x", x);
  c.flat(false, "w", w, (size_t)d.D * d.W * 4, true);
  c.flat(false, "bias", bias, (size_t)d.D * 4, false);
  c.flat(false, "cu_seqlens", cu_seqlens, ((size_t)d.B + 1) * 4, d.packed, 4);
  c.flat(false, "x0", x0, state, false);
  c.rows(true, a.y, "y", y);
  c.flat(true, "x_L", x_L, state, true);
  if ((rc = c.check())) return rc;
  a.w = w; a.bias = bias; a.cu = cu_seqlens; a.x0 = x0; a.xL = x_L;
  a.B = d.B; a.L = d.L; a.D = d.D; a.W = d.W; a.silu = d.silu;
  a.strips = (d.L + pdscan::kCvRows - 1) / pdscan::kCvRows;
  return launched(pdscan::launch_conv_fwd(a, d.in_dtype == PDSSM_BF16, (hipStream_t)stream));
}

int pdssm_conv_bwd_workspace_bytes(const pdssm_conv_dims* dims, size_t* bytes) {
  const int rc = check_conv(dims, false);
  return rc ? rc : answer(bytes, conv_ws(dims));
}

int pdssm_conv_bwd(const pdssm_conv_dims* dims, const pdssm_view* x, const float* w, const float* bias,
                   const int32_t* cu_seqlens, const void* x0, const pdssm_view* g_y, const void* g_xL,
                   const pdssm_view* g_x, float* g_w, float* g_bias, void* g_x0, void* workspace,
                   size_t workspace_bytes, void* stream) {
  int rc = check_conv(dims, false);
  if (rc || (rc = check_packed(dims->packed, cu_seqlens))) return rc;
  const pdssm_conv_dims& d = *dims;
  const CvWs n = conv_ws(dims);
  CvArgs a = {};
  Args c;
  c.es = d.in_dtype == PDSSM_BF16 ? 2 : 4;
  c.B = d.packed ? 1 : d.B; c.L = d.L; c.D = d.D;
  const size_t state = (size_t)d.B * (d.W - 1) * d.D * c.es;
  c.rows(false, a.x, "x", x);
  c.flat(false, "w", w, (size_t)d.D * d.W * 4, true);
  c.flat(false, "bias", bias, (size_t)d.D * 4, false);
  c.flat(false, "cu_seqlens", cu_seqlens, ((size_t)d.B + 1) * 4, d.packed, 4);
  c.flat(false, "x0", x0, state, false);
  c.rows(false, a.gy, "g_y", g_y);
  c.flat(false, "g_xL", g_xL, state, false);
  c.rows(true, a.gx, "g_x", g_x);
  c.flat(true, "g_w", g_w, (size_t)d.D * d.W * 4, true);
  c.flat(true, "g_bias", g_bias, (size_t)d.D * 4, true);
  c.flat(true, "g_x0", g_x0, state, false);
  if ((rc = c.check(workspace, workspace_bytes, n.total))) return rc;
  unsigned char* ws = (unsigned char*)workspace;
  a.w = w; a.bias = bias; a.cu = cu_seqlens; a.x0 = x0; a.gxL = g_xL; a.gx0 = g_x0;
  a.B = d.B; a.L = d.L; a.D = d.D; a.W = d.W; a.silu = d.silu;
  a.strips = n.strips;
  a.parts = n.parts;
  a.part = (float*)(ws + n.part);
  a.header = (uint32_t*)ws;
  const hipStream_t st = (hipStream_t)stream;
  hipError_t e = pdscan::launch_conv_bwd(a, d.in_dtype == PDSSM_BF16, st);
  SsSumArgs s = {};
  s.part = a.part;
  s.mid = (float*)(ws + n.mid);
  s.out[0] = g_w;
  s.out[1] = g_bias;
  s.share[0] = (int64_t)d.D * d.W;
  s.share[1] = d.D;
  s.parts = n.parts;
  s.width = n.width;
  if (e == hipSuccess) e = pdscan::launch_ssm_sum(s, st);
  return launched(e);
}

int pdssm_conv_step(const pdssm_conv_dims* dims, const pdssm_view* x, const float* w, const float* bias,
                    const int32_t* state_idx, int32_t n_slots, void* state, const pdssm_view* y, void* stream) {
  int rc = check_conv(dims, true);
  if (rc) return rc;
  const pdssm_conv_dims& d = *dims;
  if ((rc = check_slots(d.B, state_idx, n_slots, (int64_t)(d.W - 1) * d.D))) return rc;
  pdscan::CvStepArgs a = {};
  Args c;
  c.es = d.in_dtype == PDSSM_BF16 ? 2 : 4;
  c.B = d.B; c.L = 1; c.D = d.D;
  c.rows(false, a.x, "x", x);
  c.flat(false, "w", w, (size_t)d.D * d.W * 4, true);
  c.flat(false, "bias", bias, (size_t)d.D * 4, false);
  c.flat(false, "state_idx", state_idx, (size_t)d.B * 4, false, 4);
  c.rows(true, a.y, "y", y);
  c.flat(true, "state", state, (size_t)n_slots * (d.W - 1) * d.D * c.es, true);
  if ((rc = c.check())) return rc;
  a.w = w; a.bias = bias; a.state = state; a.idx = state_idx;
  a.B = d.B; a.D = d.D; a.W = d.W; a.silu = d.silu; a.slots = n_slots;
  return launched(pdscan::launch_conv_step(a, d.in_dtype == PDSSM_BF16, (hipStream_t)stream));
}

int pdssm_selscan_workspace_bytes(const pdssm_selscan_dims* dims, size_t* bytes) {
  int rc = check_scan(dims, false);
  if (rc) return rc;
  const ScanWs w = scan_ws(dims);
  return (rc = scan_grid(dims, w.split)) ? rc : answer(bytes, w);
}

int pdssm_selscan_bwd_workspace_bytes(const pdssm_selscan_dims* dims, size_t* bytes) {
  int rc = check_scan(dims, false);
  if (rc) return rc;
  const ScanWs w = scan_bwd_ws(dims);
  return (rc = scan_grid(dims, w.split)) ? rc : answer(bytes, w);
}

int pdssm_selscan_fwd(const pdssm_selscan_dims* dims, const pdssm_view* x, const pdssm_view* dt, const float* A,
                      const pdssm_view* Bm, const pdssm_view* Cm, const float* skip, const pdssm_view* z,
                      const float* dt_bias, const int32_t* cu_seqlens, const float* h0, const pdssm_view* y,
                      float* h_L, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_scan(dims, false);
  if (rc || (rc = check_packed(dims->packed, cu_seqlens))) return rc;
  const pdssm_selscan_dims& d = *dims;
  const ScanWs w = scan_ws(dims);
  if ((rc = scan_grid(dims, w.split))) return rc;
  const size_t state = (size_t)d.B * d.D * d.N * 4;
  SsArgs a = {};
  Args c;
  scan_in(c, a, dims, ScanIn{x, dt, Bm, Cm, z, A, skip, dt_bias});
  c.flat(false, "cu_seqlens", cu_seqlens, ((size_t)d.B + 1) * 4, d.packed, 4);
  c.flat(false, "h0", h0, state, false);
  c.rows(true, a.y, "y", y);
  c.flat(true, "h_L", h_L, state, true);
  if ((rc = c.check(workspace, workspace_bytes, w.total))) return rc;
  a.h0 = h0;
  a.hL = h_L;
  const hipStream_t st = (hipStream_t)stream;
  unsigned char* ws = (unsigned char*)workspace;
  const int bf16 = d.in_dtype == PDSSM_BF16;
  hipError_t e = scan_states(a, dims, w, cu_seqlens, ws, workspace_bytes, false, st);
  if (e == hipSuccess) e = pdscan::launch_selscan_fwd(a, bf16, st);
  return launched(e);
}

int pdssm_selscan_bwd(const pdssm_selscan_dims* dims, const pdssm_view* x, const pdssm_view* dt, const float* A,
                      const pdssm_view* Bm, const pdssm_view* Cm, const float* skip, const pdssm_view* z,
                      const float* dt_bias, const int32_t* cu_seqlens, const float* h0, const pdssm_view* g_y,
                      const float* g_hL, const pdssm_view* g_x, const pdssm_view* g_dt, float* g_A,
                      const pdssm_view* g_B, const pdssm_view* g_C, float* g_skip, const pdssm_view* g_z,
                      float* g_bias, float* g_h0, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_scan(dims, false);
  if (rc || (rc = check_packed(dims->packed, cu_seqlens))) return rc;
  const pdssm_selscan_dims& d = *dims;
  const ScanWs w = scan_bwd_ws(dims);
  if ((rc = scan_grid(dims, w.split))) return rc;
  const size_t state = (size_t)d.B * d.D * d.N * 4;
  SsArgs a = {};
  Args c;
  LaView gB, gC;
  scan_in(c, a, dims, ScanIn{x, dt, Bm, Cm, z, A, skip, dt_bias});
  c.flat(false, "cu_seqlens", cu_seqlens, ((size_t)d.B + 1) * 4, d.packed, 4);
  c.flat(false, "h0", h0, state, false);
  c.rows(false, a.gy, "g_y", g_y);
  c.flat(false, "g_hL", g_hL, state, false);
  c.rows(true, a.gx, "g_x", g_x);
  c.rows(true, a.gdt, "g_dt", g_dt);
  c.flat(true, "g_A", g_A, (size_t)d.D * d.N * 4, true);
  c.view(true, gB, "g_B", g_B, true, d.G, d.N);
  c.view(true, gC, "g_C", g_C, true, d.G, d.N);
  c.flat(true, "g_skip", g_skip, (size_t)d.D * 4, true);
  if (!c.rc && !z && g_z) c.rc = set_error(PDSSM_EINVAL, "g_z given without z");
  c.rows(true, a.gz, "g_z", g_z, z != nullptr);
  c.flat(true, "g_bias", g_bias, (size_t)d.D * 4, true);
  c.flat(true, "g_h0", g_h0, state, false);
  if ((rc = c.check(workspace, workspace_bytes, w.total))) return rc;
  a.h0 = h0;
  a.ghL = g_hL;
  a.gh0 = g_h0;
  const hipStream_t st = (hipStream_t)stream;
  unsigned char* ws = (unsigned char*)workspace;
  const int bf16 = d.in_dtype == PDSSM_BF16;
  a.ckpt = (float*)(ws + w.ckpt);
  a.cum = (float*)(ws + w.cum);
  a.part = (float*)(ws + w.part);
  a.partA = (float*)(ws + w.partA);
  hipError_t e = scan_states(a, dims, w, cu_seqlens, ws, workspace_bytes, true, st);
  if (e == hipSuccess) e = pdscan::launch_selscan_bwd(a, bf16, st);
  pdscan::SsFoldArgs f = {};
  f.part = a.part;
  f.out[0] = gB;
  f.out[1] = gC;
  f.cu = cu_seqlens;
  f.B = d.B; f.L = d.L; f.N = d.N; f.G = d.G; f.blocks = w.blocks;
  f.rows = a.rows;
  f.sum.part = a.partA;
  f.sum.mid = (float*)(ws + w.mid);
  f.sum.parts = w.split.segs;
  f.sum.width = (int64_t)d.D * (d.N + 2);
  f.sum.out[0] = g_A;
  f.sum.out[1] = g_skip;
  f.sum.out[2] = g_bias;
  f.sum.share[0] = (int64_t)d.D * d.N;
  f.sum.share[1] = f.sum.share[2] = d.D;
  if (e == hipSuccess) e = pdscan::launch_selscan_fold(f, bf16, st);
  return launched(e);
}

int pdssm_selscan_step(const pdssm_selscan_dims* dims, const pdssm_view* x, const pdssm_view* dt, const float* A,
                       const pdssm_view* Bm, const pdssm_view* Cm, const float* skip, const pdssm_view* z,
                       const float* dt_bias, const int32_t* state_idx, int32_t n_slots, float* state,
                       const pdssm_view* y, void* stream) {
  int rc = check_scan(dims, true);
  if (rc) return rc;
  const pdssm_selscan_dims& d = *dims;
  if ((rc = check_slots(d.B, state_idx, n_slots, (int64_t)d.D * d.N))) return rc;
  if ((int64_t)d.B * ((d.D + 15) / 16) > kMost)
    return set_error(PDSSM_EUNSUPPORTED, "B=%d rows of D=%d channels are too many", d.B, d.D);
  SsArgs i = {};
  pdscan::SsStepArgs a = {};
  Args c;
  scan_in(c, i, dims, ScanIn{x, dt, Bm, Cm, z, A, skip, dt_bias});
  c.flat(false, "state_idx", state_idx, (size_t)d.B * 4, false, 4);
  c.rows(true, a.y, "y", y);
  c.flat(true, "state", state, (size_t)n_slots * d.D * d.N * 4, true);
  if ((rc = c.check())) return rc;
  a.x = i.x; a.dt = i.dt; a.z = i.z; a.Bm = i.Bm; a.Cm = i.Cm;
  a.A = A; a.skip = skip; a.bias = dt_bias;
  a.state = state;
  a.idx = state_idx;
  a.B = d.B; a.D = d.D; a.N = d.N; a.G = d.G; a.slots = n_slots; a.softplus = d.softplus;
  return launched(pdscan::launch_selscan_step(a, d.in_dtype == PDSSM_BF16, (hipStream_t)stream));
}

int pdssm_norm_fwd(const pdssm_norm_dims* dims, const pdssm_view* x, const float* w, const pdssm_view* z,
                   const pdssm_view* residual, const float* res_scale, const pdssm_view* y, void* stream) {
  int rc = check_norm(dims);
  if (rc) return rc;
  const pdssm_norm_dims& d = *dims;
  NmArgs a = {};
  Args c;
  norm_in(c, a, dims, x, w, z, res_scale);
  c.view(false, a.r, "residual", residual, false, d.H, d.d);
  c.view(true, a.y, "y", y, true, d.H, d.d);
  if ((rc = c.check())) return rc;
  const int bf16 = d.in_dtype == PDSSM_BF16;
  pdscan::nm_plan(a, bf16, norm_near(dims, x), 4, 0);
  if ((int64_t)a.tiles * a.chunks > kMost) return set_error(PDSSM_EUNSUPPORTED, "too many rows and heads");
  return launched(pdscan::launch_norm_fwd(a, bf16, (hipStream_t)stream));
}

int pdssm_norm_bwd_workspace_bytes(const pdssm_norm_dims* dims, size_t* bytes) {
  const int rc = check_norm(dims);
  return rc ? rc : answer(bytes, norm_ws(dims));
}

int pdssm_norm_bwd(const pdssm_norm_dims* dims, const pdssm_view* x, const float* w, const pdssm_view* z,
                   const float* res_scale, const pdssm_view* g_y, const pdssm_view* g_x, float* g_w,
                   const pdssm_view* g_z, float* g_res_scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_norm(dims);
  if (rc) return rc;
  const pdssm_norm_dims& d = *dims;
  const NormWs n = norm_ws(dims);
  const size_t wide = (size_t)(d.per_head ? d.H : 1) * d.d * 4;
  NmArgs a = {};
  Args c;
  norm_in(c, a, dims, x, w, z, res_scale);
  c.view(false, a.gy, "g_y", g_y, true, d.H, d.d);
  c.view(true, a.gx, "g_x", g_x, true, d.H, d.d);
  c.flat(true, "g_w", g_w, wide, true);
  if (!c.rc && !z && g_z) c.rc = set_error(PDSSM_EINVAL, "g_z given without a gate");
  c.view(true, a.gz, "g_z", g_z, z != nullptr, d.H, d.d);
  if (!c.rc && !res_scale && g_res_scale) c.rc = set_error(PDSSM_EINVAL, "g_res_scale given without res_scale");
  c.flat(true, "g_res_scale", g_res_scale, wide, res_scale != nullptr);
  if ((rc = c.check(workspace, workspace_bytes, n.total))) return rc;
  const int bf16 = d.in_dtype == PDSSM_BF16;
  unsigned char* ws = (unsigned char*)workspace;
  pdscan::nm_plan(a, bf16, norm_near(dims, x), 1, norm_most(dims));
  a.part = (float*)(ws + n.part);
  a.header = (uint32_t*)ws;
  // heads with weights of their own: parts are chunks, [w of all heads][s of all]; else chunks and heads, [w][s]
  const int64_t both = res_scale ? 2 : 1, all = (int64_t)d.H * d.d;
  a.part_chunk = both * all;
  a.part_head = d.per_head ? d.d : both * d.d;
  a.part_s = d.per_head ? all : d.d;
  const hipStream_t st = (hipStream_t)stream;
  hipError_t e = pdscan::launch_norm_bwd(a, bf16, st);
  SsSumArgs s = {};
  s.part = a.part;
  s.mid = (float*)(ws + n.mid);
  s.parts = d.per_head ? a.chunks : a.chunks * d.H;
  s.share[0] = s.share[1] = d.per_head ? all : d.d;
  s.width = both * s.share[0];
  s.out[0] = g_w;
  s.out[1] = g_res_scale;
  if (e == hipSuccess) e = pdscan::launch_ssm_sum(s, st);
  return launched(e);
}

}  // extern "C"
