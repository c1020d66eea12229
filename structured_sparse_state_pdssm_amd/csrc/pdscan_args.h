// Checks of arguments that the C ABI's entry points share (host only): what
// an argument spans, its alignment and strides, and what may not overlap.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "pdscan.h"
#include "pdscan_error.h"
#include "pdscan_linattn_plan.h"

namespace pdscan {

// An argument as the elements it spans: `rows` of `bytes` each, strided over
// up to three axes (strides in bytes; axes of one element dropped).
struct Span {
  const char* name;
  const char* p;
  int64_t bytes;                 // of one row
  int64_t ext[3], str[3];        // batch, head, step
  int64_t end() const {          // one past the last byte, relative to p
    int64_t e = bytes;
    for (int i = 0; i < 3; ++i) e += (ext[i] - 1) * str[i];
    return e;
  }
};

inline Span dense(const char* name, const void* p, size_t bytes) {
  return Span{name, (const char*)p, (int64_t)bytes, {1, 1, 1}, {0, 0, 0}};
}

// Whether two arguments share a byte, as far as their spans tell: slices of
// one row-interleaved tensor (equal outer strides, rows side by side inside
// one period of them) are told apart, anything subtler counts as shared.
inline bool shared(const Span& a, const Span& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  if (!(a0 < b0 + (uintptr_t)b.end() && b0 < a0 + (uintptr_t)a.end())) return false;
  const Span& lo = a0 <= b0 ? a : b;
  const Span& hi = a0 <= b0 ? b : a;
  const int64_t gap = hi.p - lo.p;
  // the axes that both walk with one stride, from the widest stride down
  for (int64_t period : {lo.str[0], lo.str[1], lo.str[2]}) {
    if (period <= 0) continue;
    int64_t in_lo = lo.bytes, in_hi = hi.bytes;   // what lies inside one period
    bool same = true;
    for (int i = 0; i < 3; ++i) {
      const bool out_lo = lo.ext[i] > 1 && lo.str[i] >= period, out_hi = hi.ext[i] > 1 && hi.str[i] >= period;
      if (out_lo != out_hi || (out_lo && (lo.str[i] != hi.str[i] || lo.str[i] % period))) same = false;
      if (!out_lo) in_lo += (lo.ext[i] - 1) * lo.str[i];
      if (!out_hi) in_hi += (hi.ext[i] - 1) * hi.str[i];
    }
    if (!same) continue;
    const int64_t off = gap % period;
    if (off >= in_lo && off + in_hi <= period) return false;
  }
  return true;
}

// Rows of one output that share bytes with each other (a zero or short stride).
inline bool self_shared(const Span& a) {
  int64_t span = a.bytes;
  bool used[3] = {false, false, false};
  for (int n = 0; n < 3; ++n) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && a.ext[i] > 1 && (at < 0 || a.str[i] < a.str[at])) at = i;
    if (at < 0) return false;
    used[at] = true;
    if (a.str[at] < span) return true;
    span = a.str[at] * (a.ext[at] - 1) + span;
  }
  return false;
}

// A strided argument of ext[0] x ext[1] x ext[2] rows of `width` elements of
// `es` bytes: required, aligned, its strides as the loads need them.
inline int view_span(Span& s, LaView& v, const char* name, const pdssm_view* a, const int64_t* ext, int width, int es) {
  if (!a || !a->data) return set_error(PDSSM_EINVAL, "%s is NULL", name);
  const int64_t str[3] = {a->stride_b, a->stride_h, a->stride_t};
  v.p = a->data;
  s = Span{name, (const char*)a->data, (int64_t)width * es, {ext[0], ext[1], ext[2]}, {0, 0, 0}};
  if (width > 1 && ((uintptr_t)a->data & 15)) return set_error(PDSSM_EINVAL, "%s is not 16-byte aligned", name);
  if ((uintptr_t)a->data & 3) return set_error(PDSSM_EINVAL, "%s is not 4-byte aligned", name);
  for (int i = 0; i < 3; ++i) {
    if (ext[i] == 1) continue;   // an axis of one element has no step
    // three such axes stay within 64 bits of bytes
    if (str[i] < 0 || str[i] > (1ll << 40) || str[i] > (1ll << 60) / (es * (ext[i] - 1))) return set_error(PDSSM_EINVAL, "%s has a negative or huge stride", name);
    if (width > 1 && (str[i] * es) % 16)
      return set_error(PDSSM_EINVAL, "%s has a stride of %lld elements, not a multiple of 16 bytes", name,
                       (long long)str[i]);
    if (width > 1 && i == 2 && str[i] > kLaMaxStep)
      return set_error(PDSSM_EUNSUPPORTED, "%s has a step stride of %lld elements, above %d", name, (long long)str[i],
                       kLaMaxStep);
    s.str[i] = str[i] * es;
  }
  v.sb = s.str[0] / es;
  v.sh = s.str[1] / es;
  v.st = s.str[2] / es;
  return PDSSM_OK;
}

inline int dense_ok(const Span& s, bool required, uintptr_t align) {
  if (!s.p) return required ? set_error(PDSSM_EINVAL, "%s is NULL", s.name) : PDSSM_OK;
  if ((uintptr_t)s.p & (align - 1))
    return set_error(PDSSM_EINVAL, "%s is not %d-byte aligned", s.name, (int)align);
  return PDSSM_OK;
}

inline int check_overlap(const Span* in, int nin, const Span* out, int nout) {
  for (int q = 0; q < nout; ++q) {
    if (out[q].p && self_shared(out[q])) return set_error(PDSSM_EINVAL, "rows of output %s overlap", out[q].name);
    for (int r = 0; r < nin; ++r)
      if (shared(out[q], in[r]))
        return set_error(PDSSM_EINVAL, "output %s overlaps input %s", out[q].name, in[r].name);
    for (int r = q + 1; r < nout; ++r)
      if (shared(out[q], out[r]))
        return set_error(PDSSM_EINVAL, "outputs %s and %s overlap", out[q].name, out[r].name);
  }
  return PDSSM_OK;
}

inline int launched(hipError_t e) {
  if (e != hipSuccess) return set_error(PDSSM_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
  clear_error();
  return PDSSM_OK;
}

}  // namespace pdscan
