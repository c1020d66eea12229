// C ABI of the linear-attention passes (pdssm_linattn_*): argument validation
// (host only, before any HIP call), workspace layout and the order of the
// launches.  The contract of every entry point is in include/pdscan.h.

#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pdscan.h"
#include "pdscan_args.h"
#include "pdscan_error.h"
#include "pdscan_linattn_launch.h"
#include "pdscan_linattn_plan.h"

namespace {

constexpr int kCus = 256;        // compute units of the card

using pdscan::LaArgs;
using pdscan::LaJob;
using pdscan::LaSplit;
using pdscan::LaView;
using pdscan::Span;
using pdscan::check_overlap;
using pdscan::dense;
using pdscan::dense_ok;
using pdscan::launched;
using pdscan::set_error;

int check_dims(const pdssm_linattn_dims* d, bool step) {
  if (!d) return set_error(PDSSM_EINVAL, "dims is NULL");
  if (d->B < 1 || d->H < 1 || d->Hk < 1 || d->L < 1 || d->dk < 1 || d->dv < 1)
    return set_error(PDSSM_EINVAL, "dims must be >= 1 (B=%d H=%d Hk=%d L=%d dk=%d dv=%d)", d->B, d->H, d->Hk, d->L,
                     d->dk, d->dv);
  if (d->H % d->Hk) return set_error(PDSSM_EINVAL, "H=%d is not a multiple of Hk=%d", d->H, d->Hk);
  if (d->in_dtype != PDSSM_F32 && d->in_dtype != PDSSM_BF16)
    return set_error(PDSSM_EINVAL, "in_dtype must be PDSSM_F32 or PDSSM_BF16 (got %d)", d->in_dtype);
  if (d->packed != 0 && d->packed != 1) return set_error(PDSSM_EINVAL, "packed must be 0 or 1 (got %d)", d->packed);
  if (d->decay_per_head != 0 && d->decay_per_head != 1)
    return set_error(PDSSM_EINVAL, "decay_per_head must be 0 or 1 (got %d)", d->decay_per_head);
  if (!std::isfinite(d->scale)) return set_error(PDSSM_EINVAL, "scale is not finite");
  if (d->dk % 8 || d->dv % 8 || d->dk > pdscan::kLaMaxD || d->dv > pdscan::kLaMaxD)
    return set_error(PDSSM_EUNSUPPORTED, "dk=%d and dv=%d must be multiples of 8, at most %d", d->dk, d->dv,
                     pdscan::kLaMaxD);
  if (step && (d->L != 1 || d->packed))
    return set_error(PDSSM_EINVAL, "a step has L=1 and packed=0 (got L=%d packed=%d)", d->L, d->packed);
  if (d->L > 0x7fffff00) return set_error(PDSSM_EUNSUPPORTED, "L=%d is too long", d->L);
  const uint64_t units = (uint64_t)d->B * d->H;
  // (packed: L counts the rows of all sequences)
  if (units > 0x7fffffffull || (uint64_t)(d->packed ? 1 : d->B) * d->H * d->L > (1ull << 40))
    return set_error(PDSSM_EUNSUPPORTED, "B*H or the heads' rows are too many");
  return PDSSM_OK;
}

int view_span(Span& s, LaView& v, const char* name, const pdssm_view* a, const pdssm_linattn_dims* d, int heads,
              int width, int es) {
  const int64_t ext[3] = {d->packed ? 1 : d->B, heads, d->L};
  return pdscan::view_span(s, v, name, a, ext, width, es);
}

int decay_span(Span& s, LaView& v, const char* name, const pdssm_view* a, const pdssm_linattn_dims* d) {
  pdssm_view one;
  if (a && d->decay_per_head) {
    one.data = a->data;
    one.stride_b = one.stride_t = 0;
    one.stride_h = 1;
    a = &one;
  }
  return view_span(s, v, name, a, d, d->H, 1, 4);
}

struct FwdWs {
  LaSplit split;
  size_t table, starts, seg, decay, total;   // byte offsets
};

FwdWs fwd_ws(const pdssm_linattn_dims* d) {
  FwdWs w;
  const int bf16 = d->in_dtype == PDSSM_BF16;
  w.split = pdscan::la_split(d->B, d->L, d->packed, (long long)d->H * pdscan::la_slabs(d->dk, d->dv, bf16),
                             kCus * pdscan::la_resident(d->dk, d->dv, bf16, 0), (long long)d->dk * d->dv,
                             (2 * d->dk + 2 * d->dv) * (bf16 ? 2 : 4), 0x7fffff00);
  size_t at = pdscan::kLaHeader;
  auto put = [&](size_t bytes) {
    const size_t here = at;
    at += pdscan::la_align(bytes);
    return here;
  };
  const size_t units = (size_t)w.split.segs * d->H;
  w.table = w.starts = w.seg = w.decay = at;
  if (w.split.split) {
    if (d->packed) {
      w.table = put((size_t)w.split.segs * 16);
      w.starts = put(((size_t)d->B + 1) * 4);
    }
    w.seg = put(units * d->dk * d->dv * 4);
    w.decay = put(units * 4);
  }
  w.total = at;
  return w;
}

struct BwdWs {
  LaSplit split;
  size_t table, starts, segS, segR, decS, decR, r, k, xd, part, fq, fk, total;
  bool one;                      // all three jobs have one shape
  int qslabs, vslabs;            // slabs of the passes whose outputs are dk and dv wide
};

BwdWs bwd_ws(const pdssm_linattn_dims* d) {
  BwdWs w;
  const int bf16 = d->in_dtype == PDSSM_BF16;
  w.qslabs = pdscan::la_slabs(d->dv, d->dk, bf16);
  w.vslabs = pdscan::la_slabs(d->dk, d->dv, bf16);
  w.one = pdscan::la_one(d->dk, d->dv, bf16);
  // the launch with the most work decides: all three jobs in one, or those of q and k
  w.split = pdscan::la_split(d->B, d->L, d->packed, (long long)d->H * (w.one ? 3 : 2) * w.qslabs,
                             kCus * pdscan::la_resident(d->dv, d->dk, bf16, 1), 2ll * d->dk * d->dv,
                             (8 * d->dk + 7 * d->dv) * (bf16 ? 2 : 4), pdscan::kLaPiece);
  size_t at = pdscan::kLaHeader;
  auto put = [&](size_t bytes) {
    const size_t here = at;
    at += pdscan::la_align(bytes);
    return here;
  };
  const size_t units = (size_t)w.split.segs * d->H;
  const size_t rows = (size_t)(d->packed ? 1 : d->B) * d->L;
  w.table = w.starts = w.segS = w.segR = w.decS = w.decR = at;
  if (w.split.split) {
    if (d->packed) {
      w.table = put((size_t)w.split.segs * 16);
      w.starts = put(((size_t)d->B + 1) * 4);
    }
    w.segS = put(units * d->dk * d->dv * 4);
    w.segR = put(units * d->dk * d->dv * 4);
    w.decS = put(units * 4);
    w.decR = put(units * 4);
  }
  w.r = put((size_t)w.qslabs * d->H * rows * 4);
  w.k = put((size_t)w.qslabs * d->H * rows * 4);
  w.xd = put(units * w.qslabs * 8);
  w.part = put(d->decay_per_head ? units * 8 : 0);
  w.fq = w.fk = at;
  if (d->Hk != d->H) {
    w.fq = put(rows * d->H * d->dk * 4);
    w.fk = put(rows * d->H * d->dk * 4);
  }
  w.total = at;
  return w;
}

int grid_ok(const LaSplit& s, const pdssm_linattn_dims* d) {
  // workgroups are numbered in 31 bits: up to three jobs of two slabs each
  if ((uint64_t)s.segs * d->H * 6 > 0x7fffffffull)
    return set_error(PDSSM_EUNSUPPORTED, "too many segments and heads (%d, %d)", s.segs, d->H);
  return PDSSM_OK;
}

LaArgs common(const pdssm_linattn_dims* d, const LaView& g, const int32_t* cu, const LaSplit& s, unsigned char* ws,
              size_t table) {
  LaArgs a = {};
  a.g = g;
  a.cu = cu;
  a.table = (cu && s.split) ? (const int32_t*)(ws + table) : nullptr;
  a.header = (uint32_t*)ws;
  a.B = d->B; a.H = d->H; a.L = d->L;
  a.nseg = s.nseg; a.seg = s.seg; a.segs = s.segs;
  a.rows = (long long)(d->packed ? 1 : d->B) * d->L;
  a.state = (long long)d->dk * d->dv;
  return a;
}

}  // namespace

extern "C" {

int pdssm_linattn_workspace_bytes(const pdssm_linattn_dims* dims, size_t* bytes) {
  int rc = check_dims(dims, false);
  if (rc) return rc;
  if (!bytes) return set_error(PDSSM_EINVAL, "bytes is NULL");
  const FwdWs w = fwd_ws(dims);
  if ((rc = grid_ok(w.split, dims))) return rc;
  *bytes = w.total;
  pdscan::clear_error();
  return PDSSM_OK;
}

int pdssm_linattn_bwd_workspace_bytes(const pdssm_linattn_dims* dims, size_t* bytes) {
  int rc = check_dims(dims, false);
  if (rc) return rc;
  if (!bytes) return set_error(PDSSM_EINVAL, "bytes is NULL");
  const BwdWs w = bwd_ws(dims);
  if ((rc = grid_ok(w.split, dims))) return rc;
  *bytes = w.total;
  pdscan::clear_error();
  return PDSSM_OK;
}

int pdssm_linattn_fwd(const pdssm_linattn_dims* dims, const pdssm_view* q, const pdssm_view* k, const pdssm_view* v,
                      const pdssm_view* log_decay, const int32_t* cu_seqlens, const float* h0, const pdssm_view* o,
                      float* h_L, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_dims(dims, false);
  if (rc) return rc;
  const pdssm_linattn_dims& d = *dims;
  const int es = d.in_dtype == PDSSM_BF16 ? 2 : 4;
  const size_t state = (size_t)d.B * d.H * d.dk * d.dv * 4;
  const FwdWs w = fwd_ws(dims);
  if ((rc = grid_ok(w.split, dims))) return rc;
  Span in[6], out[3];
  LaView vq, vk, vv, vg, vo;
  if ((rc = view_span(in[0], vq, "q", q, dims, d.Hk, d.dk, es))) return rc;
  if ((rc = view_span(in[1], vk, "k", k, dims, d.Hk, d.dk, es))) return rc;
  if ((rc = view_span(in[2], vv, "v", v, dims, d.H, d.dv, es))) return rc;
  if ((rc = decay_span(in[3], vg, "log_decay", log_decay, dims))) return rc;
  in[4] = dense("cu_seqlens", cu_seqlens, ((size_t)d.B + 1) * 4);
  in[5] = dense("h0", h0, state);
  if ((rc = view_span(out[0], vo, "o", o, dims, d.H, d.dv, es))) return rc;
  out[1] = dense("h_L", h_L, state);
  out[2] = dense("workspace", workspace, w.total);
  if (!d.packed && cu_seqlens) return set_error(PDSSM_EINVAL, "cu_seqlens given with packed = 0");
  if ((rc = dense_ok(in[4], d.packed, 4)) || (rc = dense_ok(in[5], false, 16)) || (rc = dense_ok(out[1], true, 16)) ||
      (rc = dense_ok(out[2], true, 16)))
    return rc;
  if (workspace_bytes < w.total)
    return set_error(PDSSM_EWORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, w.total);
  if ((rc = check_overlap(in, 6, out, 3))) return rc;

  const hipStream_t st = (hipStream_t)stream;
  unsigned char* ws = (unsigned char*)workspace;
  const int bf16 = d.in_dtype == PDSSM_BF16, ratio = d.H / d.Hk;
  LaArgs a = common(dims, vg, cu_seqlens, w.split, ws, w.table);
  a.slabs = pdscan::la_slabs(d.dk, d.dv, bf16);
  a.njobs = 1;
  LaJob& J = a.job[0];
  J.x = vq; J.y = vk; J.z = vv; J.o = vo;
  J.xd = J.yd = ratio;
  J.zd = J.od = J.wd = 1;
  J.DK = d.dk; J.DV = d.dv;
  J.s_user = h0;
  J.s_fin = h_L;
  J.sm = d.dv; J.sn = 1;
  J.s_out = d.scale;
  J.s_ratio = J.s_upd = 1.0f;
  hipError_t e = hipSuccess;
  if (w.split.split) {
    // contributions of the segments, then the states that enter them
    J.s_seg = J.seg_out = (float*)(ws + w.seg);
    J.seg_decay = (float*)(ws + w.decay);
    if (d.packed)
      e = pdscan::launch_linattn_table(cu_seqlens, (int32_t*)(ws + w.table), (int32_t*)(ws + w.starts), d.B, d.L,
                                       w.split.seg, w.split.segs, st);
    if (e == hipSuccess) e = pdscan::launch_linattn_form(a, bf16, pdscan::kLaPassState, st);
    pdscan::LaCarryArgs c = {};
    c.c[0].seg = J.seg_out; c.c[0].decay = J.seg_decay; c.c[0].user = h0; c.c[0].rev = 0;
    c.starts = d.packed ? (const int32_t*)(ws + w.starts) : nullptr;
    c.B = d.B; c.H = d.H; c.nseg = w.split.nseg; c.state = a.state; c.tiles = (int)((a.state + 1023) / 1024);
    if (e == hipSuccess) e = pdscan::launch_linattn_carry(c, 1, st);
  }
  if (e == hipSuccess) e = pdscan::launch_linattn_form(a, bf16, pdscan::kLaPassFwd, st);
  return launched(e);
}

int pdssm_linattn_bwd(const pdssm_linattn_dims* dims, const pdssm_view* q, const pdssm_view* k, const pdssm_view* v,
                      const pdssm_view* log_decay, const int32_t* cu_seqlens, const float* h0, const pdssm_view* g_o,
                      const float* g_hL, const pdssm_view* g_q, const pdssm_view* g_k, const pdssm_view* g_v,
                      const pdssm_view* g_log_decay, float* g_h0, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int rc = check_dims(dims, false);
  if (rc) return rc;
  const pdssm_linattn_dims& d = *dims;
  const int es = d.in_dtype == PDSSM_BF16 ? 2 : 4;
  const size_t state = (size_t)d.B * d.H * d.dk * d.dv * 4;
  const BwdWs w = bwd_ws(dims);
  if ((rc = grid_ok(w.split, dims))) return rc;
  Span in[8], out[6];
  LaView vq, vk, vv, vg, vdo, gq, gk, gv, gg;
  if ((rc = view_span(in[0], vq, "q", q, dims, d.Hk, d.dk, es))) return rc;
  if ((rc = view_span(in[1], vk, "k", k, dims, d.Hk, d.dk, es))) return rc;
  if ((rc = view_span(in[2], vv, "v", v, dims, d.H, d.dv, es))) return rc;
  if ((rc = decay_span(in[3], vg, "log_decay", log_decay, dims))) return rc;
  in[4] = dense("cu_seqlens", cu_seqlens, ((size_t)d.B + 1) * 4);
  in[5] = dense("h0", h0, state);
  if ((rc = view_span(in[6], vdo, "g_o", g_o, dims, d.H, d.dv, es))) return rc;
  in[7] = dense("g_hL", g_hL, state);
  if ((rc = view_span(out[0], gq, "g_q", g_q, dims, d.Hk, d.dk, es))) return rc;
  if ((rc = view_span(out[1], gk, "g_k", g_k, dims, d.Hk, d.dk, es))) return rc;
  if ((rc = view_span(out[2], gv, "g_v", g_v, dims, d.H, d.dv, es))) return rc;
  if ((rc = decay_span(out[3], gg, "g_log_decay", g_log_decay, dims))) return rc;
  if (d.decay_per_head) {   // one value a head: the other axes are not walked
    out[3].ext[0] = out[3].ext[2] = 1;
  }
  out[4] = dense("g_h0", g_h0, state);
  out[5] = dense("workspace", workspace, w.total);
  if (d.H != d.Hk && (long long)d.H * d.dk > pdscan::kLaMaxStep)   // partial gradients, [rows][H][dk]
    return set_error(PDSSM_EUNSUPPORTED, "H * dk = %lld above %d with shared heads", (long long)d.H * d.dk,
                     pdscan::kLaMaxStep);
  if (!d.packed && cu_seqlens) return set_error(PDSSM_EINVAL, "cu_seqlens given with packed = 0");
  if ((rc = dense_ok(in[4], d.packed, 4)) || (rc = dense_ok(in[5], false, 16)) || (rc = dense_ok(in[7], false, 16)) ||
      (rc = dense_ok(out[4], false, 16)) || (rc = dense_ok(out[5], true, 16)))
    return rc;
  if (workspace_bytes < w.total)
    return set_error(PDSSM_EWORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, w.total);
  if ((rc = check_overlap(in, 8, out, 6))) return rc;

  const hipStream_t st = (hipStream_t)stream;
  unsigned char* ws = (unsigned char*)workspace;
  const int bf16 = d.in_dtype == PDSSM_BF16, ratio = d.H / d.Hk;
  LaArgs a = common(dims, vg, cu_seqlens, w.split, ws, w.table);
  const bool fold = ratio > 1;
  auto part = [&](size_t at) {   // fp32 partial gradients, [rows][H][dk]
    LaView v;
    v.p = ws + at;
    v.sb = (int64_t)d.L * d.H * d.dk;
    v.sh = d.dk;
    v.st = (int64_t)d.H * d.dk;
    return v;
  };
  LaJob q_job = {}, k_job = {}, v_job = {};
  // dq = scale (...): the form of (do, v, k) on the states, transposed
  q_job.x = vdo; q_job.y = vv; q_job.z = vk; q_job.w = vq;
  q_job.xd = q_job.yd = 1;
  q_job.zd = q_job.wd = ratio;
  q_job.o = fold ? part(w.fq) : gq;
  q_job.DK = d.dv; q_job.DV = d.dk;
  q_job.s_user = h0;
  q_job.s_seg = (const float*)(ws + w.segS);
  q_job.xd_with = g_hL;
  q_job.xd_out = g_hL ? (double*)(ws + w.xd) : nullptr;
  q_job.dot = (float*)(ws + w.r);
  q_job.sm = 1; q_job.sn = d.dv;
  q_job.s_out = d.scale;
  q_job.s_ratio = q_job.s_upd = 1.0f;
  // dk: the reversed form of (v, do, q) on the adjoint states, transposed
  k_job.x = vv; k_job.y = vdo; k_job.z = vq; k_job.w = vk;
  k_job.xd = k_job.yd = 1;
  k_job.zd = k_job.wd = ratio;
  k_job.o = fold ? part(w.fk) : gk;
  k_job.DK = d.dv; k_job.DV = d.dk;
  k_job.s_user = g_hL;
  k_job.s_seg = (const float*)(ws + w.segR);
  k_job.dot = (float*)(ws + w.k);
  k_job.sm = 1; k_job.sn = d.dv;
  k_job.s_out = 1.0f;
  k_job.s_ratio = k_job.s_upd = d.scale;
  k_job.rev = 1;
  q_job.mode = pdscan::kLaQ;
  k_job.mode = pdscan::kLaK;
  q_job.od = k_job.od = 1;
  q_job.o_f32 = k_job.o_f32 = fold;
  // dv: the reversed form of (k, q, do)
  v_job.x = vk; v_job.y = vq; v_job.z = vdo; v_job.o = gv;
  v_job.xd = v_job.yd = ratio;
  v_job.zd = v_job.od = v_job.wd = 1;
  v_job.DK = d.dk; v_job.DV = d.dv;
  v_job.s_user = g_hL;
  v_job.s_seg = (const float*)(ws + w.segR);
  v_job.s_fin = g_h0;
  v_job.sm = d.dv; v_job.sn = 1;
  v_job.s_out = 1.0f;
  v_job.s_ratio = v_job.s_upd = d.scale;
  v_job.rev = 1;
  v_job.mode = pdscan::kLaV;

  hipError_t e = hipSuccess;
  if (w.split.split) {
    if (d.packed)
      e = pdscan::launch_linattn_table(cu_seqlens, (int32_t*)(ws + w.table), (int32_t*)(ws + w.starts), d.B, d.L,
                                       w.split.seg, w.split.segs, st);
    // states forwards from (k, v), adjoint states backwards from (q, do)
    LaArgs s = a;
    s.slabs = w.vslabs;
    s.njobs = 2;
    s.job[0] = v_job;
    s.job[0].y = vk; s.job[0].z = vv;
    s.job[0].rev = 0;
    s.job[0].s_upd = 1.0f;
    s.job[0].seg_out = (float*)(ws + w.segS);
    s.job[0].seg_decay = (float*)(ws + w.decS);
    s.job[1] = v_job;
    s.job[1].seg_out = (float*)(ws + w.segR);
    s.job[1].seg_decay = (float*)(ws + w.decR);
    if (e == hipSuccess) e = pdscan::launch_linattn_form(s, bf16, pdscan::kLaPassState, st);
    pdscan::LaCarryArgs c = {};
    c.c[0].seg = s.job[0].seg_out; c.c[0].decay = s.job[0].seg_decay; c.c[0].user = h0; c.c[0].rev = 0;
    c.c[1].seg = s.job[1].seg_out; c.c[1].decay = s.job[1].seg_decay; c.c[1].user = g_hL; c.c[1].rev = 1;
    c.starts = d.packed ? (const int32_t*)(ws + w.starts) : nullptr;
    c.B = d.B; c.H = d.H; c.nseg = w.split.nseg; c.state = a.state; c.tiles = (int)((a.state + 1023) / 1024);
    if (e == hipSuccess) e = pdscan::launch_linattn_carry(c, 2, st);
  }
  LaArgs m = a;
  m.slabs = w.qslabs;
  m.job[0] = q_job;
  m.job[1] = k_job;
  m.njobs = 2;
  if (w.one) {   // one launch: the three jobs of a segment read the same rows
    m.job[2] = v_job;
    m.njobs = 3;
  }
  if (e == hipSuccess) e = pdscan::launch_linattn_form(m, bf16, w.one ? pdscan::kLaPassQKV : pdscan::kLaPassQK, st);
  if (!w.one) {
    m.slabs = w.vslabs;
    m.job[0] = v_job;
    m.njobs = 1;
    if (e == hipSuccess) e = pdscan::launch_linattn_form(m, bf16, pdscan::kLaPassV, st);
  }
  pdscan::LaDecayArgs g = {};
  g.c = a;
  g.r = (const float*)(ws + w.r);
  g.k = (const float*)(ws + w.k);
  g.sS = (const float*)(ws + w.segS);
  g.sR = (const float*)(ws + w.segR);
  g.xd = q_job.xd_out;
  g.part = (double*)(ws + w.part);
  g.out = gg;
  g.slabs = w.qslabs;
  g.per_head = d.decay_per_head;
  g.h0 = h0;
  g.g_h0 = g_h0;
  if (e == hipSuccess) e = pdscan::launch_linattn_decay(g, st);
  if (fold) {
    pdscan::LaFoldArgs f = {};
    f.cu = cu_seqlens;
    f.B = d.B; f.H = d.H; f.L = d.L; f.ratio = ratio; f.d = d.dk; f.bf16 = bf16;
    f.rows = a.rows;
    f.part_q = (const float*)(ws + w.fq);
    f.part_k = (const float*)(ws + w.fk);
    f.out_q = gq;
    f.out_k = gk;
    if (e == hipSuccess) e = pdscan::launch_linattn_fold(f, st);
  }
  return launched(e);
}

int pdssm_linattn_step(const pdssm_linattn_dims* dims, const pdssm_view* q, const pdssm_view* k, const pdssm_view* v,
                       const pdssm_view* log_decay, const int32_t* state_idx, int32_t n_slots, float* state,
                       const pdssm_view* o, void* stream) {
  int rc = check_dims(dims, true);
  if (rc) return rc;
  const pdssm_linattn_dims& d = *dims;
  if (n_slots < 1) return set_error(PDSSM_EINVAL, "n_slots must be >= 1 (got %d)", n_slots);
  if (!state_idx && n_slots < d.B)
    return set_error(PDSSM_EINVAL, "n_slots=%d < B=%d without state_idx", n_slots, d.B);
  if ((uint64_t)n_slots * d.H > (1ull << 40)) return set_error(PDSSM_EUNSUPPORTED, "n_slots * H is too large");
  const int es = d.in_dtype == PDSSM_BF16 ? 2 : 4;
  Span in[5], out[2];
  LaView vq, vk, vv, vg, vo;
  if ((rc = view_span(in[0], vq, "q", q, dims, d.Hk, d.dk, es))) return rc;
  if ((rc = view_span(in[1], vk, "k", k, dims, d.Hk, d.dk, es))) return rc;
  if ((rc = view_span(in[2], vv, "v", v, dims, d.H, d.dv, es))) return rc;
  if ((rc = decay_span(in[3], vg, "log_decay", log_decay, dims))) return rc;
  in[4] = dense("state_idx", state_idx, (size_t)d.B * 4);
  if ((rc = view_span(out[0], vo, "o", o, dims, d.H, d.dv, es))) return rc;
  out[1] = dense("state", state, (size_t)n_slots * d.H * d.dk * d.dv * 4);
  if ((rc = dense_ok(in[4], false, 4)) || (rc = dense_ok(out[1], true, 16))) return rc;
  if ((rc = check_overlap(in, 5, out, 2))) return rc;
  pdscan::LaStepArgs a = {};
  a.q = vq; a.k = vk; a.v = vv; a.g = vg; a.o = vo;
  a.state = state;
  a.idx = state_idx;
  a.B = d.B; a.H = d.H; a.qd = d.H / d.Hk; a.dk = d.dk; a.dv = d.dv; a.slots = n_slots;
  a.scale = d.scale;
  a.bf16 = d.in_dtype == PDSSM_BF16;
  // Columns per workgroup: whole rows (16 states of 128/128 6.1 us, 264 of 16/64 4.1), halved down to 16 (64
  // bytes of a row) while there is not a workgroup for every compute unit (the 16 5.0 us; the 264 in quarters 6.8).
  a.cols = d.dv;
  while (a.cols >= 32 && a.cols % 16 == 0 && (long long)d.B * d.H * (d.dv / a.cols) < kCus) a.cols /= 2;
  if ((long long)d.B * d.H * ((d.dv + a.cols - 1) / a.cols) > 0x7fffffffll)
    return set_error(PDSSM_EUNSUPPORTED, "too many rows and heads (%d, %d)", d.B, d.H);
  return launched(pdscan::launch_linattn_step(a, (hipStream_t)stream));
}

}  // extern "C"
