// Linear attention with a decay for each head, in chunks.
//
//   S_t = a_t S_{t-1} + y_t z_t^T,   o_t = s S_t^T x_t,   a_t = exp(g_t)
//
// With G the inclusive sums of g inside a chunk of C tokens and S_in the state
// that enters it,
//   o_i   = s ( e^{G_i} S_in^T x_i + sum_{j <= i} e^{G_i - G_j} (x_i . y_j) z_j )
//   S_out = e^{G_C} S_in + sum_j e^{G_C - G_j} y_j z_j^T.
// The same form run backwards in time (j >= i, weights e^{G_j - G_i}, output
// scale e^{G_C - G_i}, update weight e^{G_j}) is the adjoint recurrence, so
// the forward pass and all three gradients are one kernel on other operands:
//   o  = form(q, k, v)      dq = form(do, v, k)                  forwards
//   dv = form(k, q, do)     dk = form(v, do, q)                  backwards.
//
// One workgroup owns one segment of a sequence, one head and 32 columns of z
// per wave; the state stays in the accumulators of its matrix instructions.
// Every exponent is a difference of sums that ends at or below zero, held as
// two floats (the sums are formed in 64 bits), so a strong decay does not
// spoil the differences behind it.
//
// Precision.  bf16 inputs enter the products as they are.  What is computed
// (the state, the weighted scores, the weighted values) is held in fp32 and
// enters a product as two or three bf16 pieces x = x0 + x1 (+ x2), each the
// next eight significant bits: two leave 2^-16 of a term (outputs in bf16
// are rounded at 2^-9), three are exact but for the last bit (the state is
// an fp32 output).  fp32 inputs use fp32 products throughout.
#pragma once

#include <hip/hip_runtime.h>

#include "pdscan_linattn_plan.h"

namespace pdscan {

typedef __bf16 la_bf8 __attribute__((ext_vector_type(8)));
typedef float la_f16 __attribute__((ext_vector_type(16)));
typedef short la_s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) la_s4 la_lds_s4;

struct LaBf16 {
  using store = uint16_t;
  static constexpr int kVec = 8;    // elements of 16 bytes
  static constexpr int kPad = 8;    // row padding in LDS: rows land 4 banks apart
  union frag {
    uint32_t u[4];
    la_s4 s[2];
    la_bf8 v;
  };
  static __device__ __forceinline__ void mma(la_f16& c, const frag& a, const frag& b) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float get(const frag& f, int e) {
    const uint32_t w = f.u[e >> 1];
    return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  // elements k0 + 4h + {0..3} and k0 + 8 + 4h + {0..3} of a row
  static __device__ __forceinline__ frag row(const store* p, int h) {
    frag f;
    *(uint2*)&f.u[0] = *(const uint2*)(p + 4 * h);
    *(uint2*)&f.u[2] = *(const uint2*)(p + 8 + 4 * h);
    return f;
  }
  // the same elements of a column: rows r0 + 4h + {0..3} and r0 + 8 + 4h + {0..3}
  // of column c0 + lane % 32.  The transposing read hands the 16 lanes of a
  // group four rows of 16 columns: lane p points at row p / 4, columns
  // 4 (p % 4).. and receives column p.
  static __device__ __forceinline__ frag col(const store* base, int stride, int r0, int c0, int lane) {
    const int p = lane & 15;
    const store* a = base + (r0 + 4 * (lane >> 5) + (p >> 2)) * stride + c0 + (lane & 16) + 4 * (p & 3);
    frag f;
    f.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((la_lds_s4*)(a));
    f.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((la_lds_s4*)(a + 8 * stride));
    return f;
  }
  // eight floats as bf16 pieces, cut (not rounded) so that each rest is exact
  template <int NP>
  static __device__ __forceinline__ void pieces(const float* v, frag* out) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v[e];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = __float_as_uint(x[2 * e]), hi = __float_as_uint(x[2 * e + 1]);
        out[p].u[e] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
        if (p + 1 < NP) {
          x[2 * e] -= __uint_as_float(lo & 0xffff0000u);
          x[2 * e + 1] -= __uint_as_float(hi & 0xffff0000u);
        }
      }
    }
  }
  template <int NP>
  static __device__ __forceinline__ void put4(store* p, int piece_stride, const float* v) {
    float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      uint2 w;
      const uint32_t b0 = __float_as_uint(x[0]), b1 = __float_as_uint(x[1]), b2 = __float_as_uint(x[2]),
                     b3 = __float_as_uint(x[3]);
      w.x = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
      w.y = __builtin_amdgcn_perm(b3, b2, 0x07060302u);
      *(uint2*)(p + q * piece_stride) = w;
      if (q + 1 < NP) {
        x[0] -= __uint_as_float(b0 & 0xffff0000u);
        x[1] -= __uint_as_float(b1 & 0xffff0000u);
        x[2] -= __uint_as_float(b2 & 0xffff0000u);
        x[3] -= __uint_as_float(b3 & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ uint32_t round(float x) {   // nearest, ties to even
    const uint32_t b = __float_as_uint(x);
    if ((b & 0x7fffffffu) > 0x7f800000u) return (b >> 16) | 0x40u;
    return (b + 0x7fffu + ((b >> 16) & 1u)) >> 16;
  }
  static __device__ __forceinline__ void store4(store* p, const float* v) {
    uint2 w;
    w.x = round(v[0]) | (round(v[1]) << 16);
    w.y = round(v[2]) | (round(v[3]) << 16);
    *(uint2*)p = w;
  }
  static __device__ __forceinline__ void load4(const store* p, float* v) {
    const uint2 w = *(const uint2*)p;
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
};

struct LaF32 {
  using store = float;
  static constexpr int kVec = 4;
  static constexpr int kPad = 4;
  struct frag {
    float f[8];
  };
  static __device__ __forceinline__ void mma(la_f16& c, const frag& a, const frag& b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.f[e], b.f[e], c, 0, 0, 0);
  }
  static __device__ __forceinline__ float get(const frag& f, int e) { return f.f[e]; }
  static __device__ __forceinline__ frag row(const store* p, int h) {
    frag f;
    *(float4*)&f.f[0] = *(const float4*)(p + 4 * h);
    *(float4*)&f.f[4] = *(const float4*)(p + 8 + 4 * h);
    return f;
  }
  static __device__ __forceinline__ frag col(const store* base, int stride, int r0, int c0, int lane) {
    const store* a = base + (r0 + 4 * (lane >> 5)) * stride + c0 + (lane & 31);
    frag f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f.f[e] = a[e * stride];
      f.f[4 + e] = a[(8 + e) * stride];
    }
    return f;
  }
  template <int NP>
  static __device__ __forceinline__ void pieces(const float* v, frag* out) {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[0].f[e] = v[e];
  }
  template <int NP>
  static __device__ __forceinline__ void put4(store* p, int, const float* v) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  }
  static __device__ __forceinline__ void store4(store* p, const float* v) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  }
  static __device__ __forceinline__ void load4(const store* p, float* v) {
    const float4 w = *(const float4*)p;
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  }
};

struct LaSeg {
  int b, vb, t0, len, first, last;   // sequence, batch index of the views, first step, steps
  long long row0;                    // first row of [rows] arrays
};

__device__ __forceinline__ bool la_segment(const LaArgs& a, int sid, LaSeg& s) {
  if (a.table) {
    const int4 e = *(const int4*)(a.table + 4 * (long long)sid);
    if (e.z < 0) return false;
    s.b = e.x; s.vb = 0; s.t0 = e.y; s.len = e.z; s.first = e.w & 1; s.last = e.w >> 1;
    s.row0 = s.t0;
  } else if (a.cu) {
    // offsets outside the token axis or out of order are cut to it: nothing is read past the rows
    int t0 = a.cu[sid], t1 = a.cu[sid + 1];
    t0 = t0 < 0 ? 0 : t0 > a.L ? a.L : t0;
    t1 = t1 < t0 ? t0 : t1 > a.L ? a.L : t1;
    s.b = sid; s.vb = 0; s.t0 = t0; s.len = t1 - t0; s.first = 1; s.last = 1;
    s.row0 = t0;
  } else {
    s.b = s.vb = sid / a.nseg;
    const int q = sid % a.nseg;
    s.t0 = q * a.seg;
    s.len = a.L - s.t0 < a.seg ? a.L - s.t0 : a.seg;
    s.first = q == 0;
    s.last = q == a.nseg - 1;
    s.row0 = (long long)s.b * a.L + s.t0;
  }
  return true;
}

template <typename T>
__device__ __forceinline__ const typename T::store* la_ptr(const LaView& v, int b, int h, int t) {
  return (const typename T::store*)v.p + (int64_t)b * v.sb + (int64_t)h * v.sh + (int64_t)t * v.st;
}

// A tile of C rows and W elements on its way from memory to LDS: thread
// `tid` owns 16 bytes of every RP-th row.  fetch() only issues the loads (the
// next chunk's while this one is worked on); rows behind n and columns behind
// D are loaded from a place that exists and become zero in commit().
template <typename T, int C, int W, int NT>
struct LaTileIO {
  using E = typename T::store;
  static constexpr int kCols = W / T::kVec, RP = NT / kCols, N = C / RP, kStride = W + T::kPad;
  uint4 r[N];
  int row0, col;
  bool ok;
  __device__ __forceinline__ void init(int tid, int D) {
    row0 = tid / kCols;
    col = tid % kCols * T::kVec;
    ok = col < D;
    if (!ok) col = 0;
  }
  __device__ __forceinline__ void fetch(const E* chunk, int64_t st, int n) {
    if (n >= C) {
      const E* p = chunk + (int64_t)row0 * st + col;
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = *(const uint4*)(p + (int64_t)(i * RP) * st);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = row0 + i * RP;
        r[i] = *(const uint4*)(chunk + (int64_t)(row < n ? row : n - 1) * st + col);
      }
    }
  }
  __device__ __forceinline__ void commit(E* lds, int tid, int n) const {
    E* q = lds + row0 * kStride + tid % kCols * T::kVec;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint4 w = r[i];
      if (!ok || row0 + i * RP >= n) w = make_uint4(0, 0, 0, 0);
      *(uint4*)(q + i * RP * kStride) = w;
    }
  }
};

__device__ __forceinline__ double la_dpp_add(double x, uint64_t up) { return x + __longlong_as_double((long long)up); }

// x plus the value of the lane that DPP control CTRL names (zero where there
// is none or the row is masked)
template <int CTRL, int ROWS>
__device__ __forceinline__ double la_scan_step(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return la_dpp_add(x, ((uint64_t)hi << 32) | lo);
}

// Exponents of one chunk, by one wave (lane = token, g = its log decay, 0
// behind the last): G as two floats in units of log 2, the output scale and
// the update weight of every token, and the chunk's whole decay behind them.
// A log decay under -1e4 (minus infinity: the state starts anew) counts as
// -1e4, whose exponential is zero all the same.  Returns the sum of log2.
template <int C>
__device__ __forceinline__ double la_exponents(float g, int rev, float s_inter, float s_upd, float* e, int lane) {
  if (g < -1e4f) g = -1e4f;
  double G = (double)g * 1.4426950408889634074;
  G = la_scan_step<0x111, 0xf>(G);   // row_shr:1
  G = la_scan_step<0x112, 0xf>(G);   // row_shr:2
  G = la_scan_step<0x114, 0xf>(G);   // row_shr:4
  G = la_scan_step<0x118, 0xf>(G);   // row_shr:8
  G = la_scan_step<0x142, 0xa>(G);   // row_bcast:15 into rows 1 and 3
  G = la_scan_step<0x143, 0xc>(G);   // row_bcast:31 into rows 2 and 3
  const uint64_t b = (uint64_t)__double_as_longlong(G);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  const double tot = __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
  if (lane < C) {
    const float gh = (float)G;
    e[lane] = gh;
    e[C + lane] = (float)(G - (double)gh);
    const float from = __builtin_amdgcn_exp2f((float)G), to = __builtin_amdgcn_exp2f((float)(tot - G));
    e[2 * C + lane] = (rev ? to : from) * s_inter;
    e[3 * C + lane] = (rev ? from : to) * s_upd;
  }
  if (lane == 0) e[4 * C] = __builtin_amdgcn_exp2f((float)tot);
  return tot;
}

template <typename T, int DKP, int NW>
struct LaTile {
  static constexpr bool kF32 = sizeof(typename T::store) == 4;
  static constexpr int C = (kF32 && DKP == 256) ? 32 : 64;
  static constexpr int NT = NW * 64;
  static constexpr int IT = C / 32;              // 32-token tiles of a chunk
  static constexpr int KT = DKP / 32;            // 32-row tiles of the state
  static constexpr int NPS = kF32 ? 1 : 3;       // pieces of the state's update
  // One or two waves form all scores of the chunk each, in registers; four
  // share them through LDS (each wave forms one tile of 32 x 32).
  static constexpr bool kShareP = NW == 4;
  static constexpr int XS = DKP + T::kPad, ZS = NW * 32 + T::kPad, PS = C + 4;
  static constexpr int kExp = 4 * C + 4;         // floats of one chunk's exponents
  static constexpr size_t kX = (size_t)C * XS * sizeof(typename T::store);
  static constexpr size_t kZ = (size_t)C * ZS * sizeof(typename T::store);
  static constexpr size_t kP = kShareP ? (size_t)C * PS * sizeof(typename T::store) : 0;
  static constexpr size_t kSmall = (size_t)(2 * kExp + NW * C) * 4;
  static constexpr size_t main_bytes(int np) { return 2 * kX + kZ + np * kP + kSmall; }
  static constexpr size_t state_bytes() { return kX + kZ + (size_t)2 * kExp * 4; }
  using X = LaTileIO<T, C, DKP, NT>;
  using Z = LaTileIO<T, C, NW * 32, NT>;
  // registers: state, outputs and the tiles under way; under about 200 of
  // them two waves share a SIMD
  static constexpr int kRegs = 16 * (KT + IT) + 4 * (2 * X::N + Z::N);
  static constexpr int kWaves = kRegs <= 180 ? 2 : 1;
};

// acc (C layout of a 32 x 32 product: column lane % 32, rows 8 (r / 4) + 4 h +
// r % 4) gives the eight contraction slots of step q of the next product: the
// operand loads above use the same order, so no lane exchanges anything.
template <typename T, int DKP, int NW>
__device__ __forceinline__ void la_update(la_f16 (&S)[DKP / 32], const typename T::store* Y,
                                          const typename T::frag* zf, const float* ew, float decay, int lane) {
  using K = LaTile<T, DKP, NW>;
  const int h = lane >> 5;
#pragma unroll
  for (int t = 0; t < K::KT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) S[t][r] *= decay;
#pragma unroll
  for (int js = 0; js < K::C / 16; ++js) {
    float v[8];
    const float4 w0 = *(const float4*)(ew + 16 * js + 4 * h), w1 = *(const float4*)(ew + 16 * js + 8 + 4 * h);
    const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = T::get(zf[js], e) * w[e];
    typename T::frag b[K::NPS];
    T::template pieces<K::NPS>(v, b);
#pragma unroll
    for (int t = 0; t < K::KT; ++t) {
      const typename T::frag y = T::col(Y, K::XS, 16 * js, 32 * t, lane);
#pragma unroll
      for (int p = 0; p < K::NPS; ++p) T::mma(S[t], y, b[p]);
    }
  }
}

// A state's rows m and column `col` of this lane, zero where p is NULL or the
// state ends.  sm = 1: the rows lie side by side (the state is stored
// transposed) and four come in one load.
template <int KT>
__device__ __forceinline__ void la_load_state(la_f16 (&S)[KT], const float* p, int sm, int sn, int DK, int DV,
                                              int col, int h) {
#pragma unroll
  for (int t = 0; t < KT; ++t) S[t] = la_f16{};
  if (!p) return;
  const float* q = p + (long long)(col < DV ? col : 0) * sn;
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int m = 32 * t + 8 * r4 + 4 * h;
      const bool in = m < DK && col < DV;
      const int mm = m < DK ? m : 0;
      float v[4];
      if (sm == 1) {
        const float4 w = *(const float4*)(q + mm);
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = q[(long long)(mm + e) * sm];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][4 * r4 + e] = in ? v[e] : 0.0f;
    }
}

template <int KT>
__device__ __forceinline__ void la_store_state(const la_f16 (&S)[KT], float* p, int sm, int sn, int DK, int DV,
                                               int col, int h) {
  if (col >= DV) return;
  float* q = p + (long long)col * sn;
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int m = 32 * t + 8 * r4 + 4 * h;
      if (m >= DK) continue;
      if (sm == 1)
        *(float4*)(q + m) = make_float4(S[t][4 * r4], S[t][4 * r4 + 1], S[t][4 * r4 + 2], S[t][4 * r4 + 3]);
      else
#pragma unroll
        for (int e = 0; e < 4; ++e) q[(long long)(m + e) * sm] = S[t][4 * r4 + e];
    }
}

// Scores of one 32 x 32 tile (rows j of y, columns i of x), weighted by the
// decay between the two tokens and zero on the wrong side of the diagonal.
template <typename T, int DKP, int NW>
__device__ __forceinline__ la_f16 la_scores(const typename T::store* X, const typename T::store* Y, const float* e,
                                            int jt, int it, int rev, float s_intra, int lane) {
  using K = LaTile<T, DKP, NW>;
  const int h = lane >> 5, n32 = lane & 31;
  la_f16 c = {};
#pragma unroll
  for (int ks = 0; ks < DKP / 16; ++ks)
    T::mma(c, T::row(Y + (32 * jt + n32) * K::XS + 16 * ks, h), T::row(X + (32 * it + n32) * K::XS + 16 * ks, h));
  const int i = 32 * it + n32;
  const float gi = e[i], gl = e[K::C + i];
  const float sign = rev ? -1.0f : 1.0f;
#pragma unroll
  for (int r4 = 0; r4 < 4; ++r4) {
    const int j0 = 32 * jt + 8 * r4 + 4 * h;
    const float4 jh = *(const float4*)(e + j0), jl = *(const float4*)(e + K::C + j0);
    const float hh[4] = {jh.x, jh.y, jh.z, jh.w}, ll[4] = {jl.x, jl.y, jl.z, jl.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float d = ((gi - hh[q]) + (gl - ll[q])) * sign;
      const float w = __builtin_amdgcn_exp2f(d) * s_intra;
      const float v = c[4 * r4 + q] * w;
      c[4 * r4 + q] = jt != it || (rev ? j0 + q >= i : j0 + q <= i) ? v : 0.0f;
    }
  }
  return c;
}

// o = form(x, y, z) over one segment, head and slab of 32 NW columns.
template <typename T, int DKP, int NW, int NP>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(LaTile<T, DKP, NW>::kWaves))) void
pdssm_linattn_kernel(const LaArgs a) {
  using K = LaTile<T, DKP, NW>;
  using E = typename T::store;
  using F = typename T::frag;
  constexpr int C = K::C, IT = K::IT;
  extern __shared__ __align__(16) unsigned char smem[];
  E* X = (E*)smem;
  E* Y = (E*)(smem + K::kX);
  E* Z = (E*)(smem + 2 * K::kX);
  E* P = (E*)(smem + 2 * K::kX + K::kZ);
  float* exps = (float*)(smem + 2 * K::kX + K::kZ + NP * K::kP);   // of this chunk and the next
  float* dots = exps + 2 * K::kExp;                                // [NW][C]

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5,
            n32 = lane & 31;
  unsigned id = blockIdx.x;
  if (id == 0 && tid < 2) a.header[tid] = 0;
  const int jn = id % a.njobs;
  id /= a.njobs;
  const int slab = id % a.slabs;
  id /= a.slabs;
  const int hd = id % a.H;
  const int sid = id / a.H;
  const LaJob& J = a.job[jn];
  LaSeg s;
  if (!la_segment(a, sid, s)) return;

  const int rev = J.rev;
  const int slab0 = slab * NW * 32;
  const int c0 = slab0 + wave * 32;      // first column of this wave
  const int col = c0 + n32;
  const long long unit = (long long)s.b * a.H + hd;
  const bool starts = rev ? s.last : s.first, ends = rev ? s.first : s.last;
  const int chunks = (s.len + C - 1) / C;
  const E* xp = la_ptr<T>(J.x, s.vb, hd / J.xd, s.t0);
  const E* yp = la_ptr<T>(J.y, s.vb, hd / J.yd, s.t0);
  const E* zp = la_ptr<T>(J.z, s.vb, hd / J.zd, s.t0) + slab0;
  const float* gp = (const float*)a.g.p + (int64_t)s.vb * a.g.sb + (int64_t)hd * a.g.sh + (int64_t)s.t0 * a.g.st;
  typename K::X tx, ty;
  typename K::Z tz;
  tx.init(tid, J.DK);
  ty.init(tid, J.DK);
  tz.init(tid, J.DV - slab0);
  float gv = 0.0f;
  constexpr int kExpWave = NW - 1;

  auto fetch = [&](int ci) {
    const int n = s.len - ci * C;
    tx.fetch(xp + (int64_t)(ci * C) * J.x.st, J.x.st, n);
    ty.fetch(yp + (int64_t)(ci * C) * J.y.st, J.y.st, n);
    tz.fetch(zp + (int64_t)(ci * C) * J.z.st, J.z.st, n);
    if (wave == kExpWave) gv = lane < n && lane < C ? gp[(int64_t)(ci * C + lane) * a.g.st] : 0.0f;
  };
  if (chunks) fetch(rev ? chunks - 1 : 0);

  const float* init = starts ? (J.s_user ? J.s_user + unit * a.state : nullptr)
                             : J.s_seg + ((long long)sid * a.H + hd) * a.state;
  la_f16 S[K::KT];
  la_load_state<K::KT>(S, init, J.sm, J.sn, J.DK, J.DV, col, h);
  if (wave == kExpWave) la_exponents<C>(gv, rev, J.s_inter, J.s_upd, exps, lane);

  for (int q = 0; q < chunks; ++q) {
    const int ci = rev ? chunks - 1 - q : q;
    const int t = s.t0 + ci * C;
    const int n = s.len - ci * C < C ? s.len - ci * C : C;
    const float* e = exps + (q & 1) * K::kExp;
    tx.commit(X, tid, n);
    ty.commit(Y, tid, n);
    tz.commit(Z, tid, n);
    __syncthreads();
    if (q + 1 < chunks) fetch(rev ? ci - 1 : ci + 1);

    if constexpr (K::kShareP) {
      static_assert(IT * IT <= NW, "a score tile per wave");
      const int jt = wave / IT, it = wave % IT;
      if (wave < IT * IT && (rev ? jt >= it : jt <= it)) {
        const la_f16 c = la_scores<T, DKP, NW>(X, Y, e, jt, it, rev, J.s_intra, lane);
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const float v[4] = {c[4 * r4], c[4 * r4 + 1], c[4 * r4 + 2], c[4 * r4 + 3]};
          T::template put4<NP>(P + (32 * it + n32) * K::PS + 32 * jt + 8 * r4 + 4 * h, C * K::PS, v);
        }
      }
    }

    // what the entering state gives
    la_f16 o[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) o[it] = la_f16{};
#pragma unroll
    for (int t4 = 0; t4 < K::KT; ++t4)
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        float v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = S[t4][8 * k2 + r];
        F sp[NP];
        T::template pieces<NP>(v, sp);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const F xb = T::row(X + (32 * it + n32) * K::XS + 32 * t4 + 16 * k2, h);
#pragma unroll
          for (int p = 0; p < NP; ++p) T::mma(o[it], sp[p], xb);
        }
      }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const float w = e[2 * C + 32 * it + n32];
#pragma unroll
      for (int r = 0; r < 16; ++r) o[it][r] *= w;
    }

    // what the chunk's own tokens give
    F zf[C / 16];
#pragma unroll
    for (int js = 0; js < C / 16; ++js) zf[js] = T::col(Z, K::ZS, 16 * js, wave * 32, lane);
    if constexpr (K::kShareP) {
      __syncthreads();
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int js = 0; js < C / 16; ++js) {
          if (rev ? js < 2 * it : js >= 2 * it + 2) continue;
#pragma unroll
          for (int p = 0; p < NP; ++p)
            T::mma(o[it], zf[js], T::row(P + p * C * K::PS + (32 * it + n32) * K::PS + 16 * js, h));
        }
    } else {
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int jt = 0; jt < IT; ++jt) {
          if (rev ? jt < it : jt > it) continue;
          const la_f16 c = la_scores<T, DKP, NW>(X, Y, e, jt, it, rev, J.s_intra, lane);
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] = c[8 * k2 + r];
            F pp[NP];
            T::template pieces<NP>(v, pp);
#pragma unroll
            for (int p = 0; p < NP; ++p) T::mma(o[it], zf[2 * jt + k2], pp[p]);
          }
        }
    }

#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int i = 32 * it + n32;
      float dsum = 0.0f;
      if (i < n) {
        const int64_t oo = (int64_t)s.vb * J.o.sb + (int64_t)(hd / J.od) * J.o.sh + (int64_t)(t + i) * J.o.st;
        const E* wp = J.dot ? la_ptr<T>(J.w, s.vb, hd / J.wd, t + i) : nullptr;
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int cc = c0 + 8 * r4 + 4 * h;
          if (cc >= J.DV) continue;
          const float v[4] = {o[it][4 * r4], o[it][4 * r4 + 1], o[it][4 * r4 + 2], o[it][4 * r4 + 3]};
          if (J.o_f32)
            *(float4*)((float*)J.o.p + oo + cc) = make_float4(v[0], v[1], v[2], v[3]);
          else
            T::store4((E*)J.o.p + oo + cc, v);
          if (wp) {
            float w[4];
            T::load4(wp + cc, w);
            dsum += (w[0] * v[0] + w[1] * v[1]) + (w[2] * v[2] + w[3] * v[3]);
          }
        }
      }
      if (J.dot) {
        dsum += __shfl_xor(dsum, 32, 64);
        if (h == 0) dots[wave * C + i] = dsum;
      }
    }

    la_update<T, DKP, NW>(S, Y, zf, e + 3 * C, e[4 * C], lane);
    if (wave == kExpWave && q + 1 < chunks)
      la_exponents<C>(gv, rev, J.s_inter, J.s_upd, exps + ((q + 1) & 1) * K::kExp, lane);
    __syncthreads();
    if (J.dot && tid < n) {
      float d = 0.0f;
      for (int w = 0; w < NW; ++w) d += dots[w * C + tid];
      J.dot[((long long)slab * a.H + hd) * a.rows + s.row0 + (t - s.t0) + tid] = d;
    }
  }

  if (!ends) return;
  if (J.s_fin) la_store_state<K::KT>(S, J.s_fin + unit * a.state, J.sm, J.sn, J.DK, J.DV, col, h);
  if (J.xd_out) {
    // final state . its gradient
    la_f16 R[K::KT];
    la_load_state<K::KT>(R, J.xd_with + unit * a.state, J.sm, J.sn, J.DK, J.DV, col, h);
    double d = 0.0;
#pragma unroll
    for (int t = 0; t < K::KT; ++t) {
      float p = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) p += S[t][r] * R[t][r];
      d += (double)p;
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) d += __shfl_xor(d, m, 64);
    double* red = (double*)smem;
    __syncthreads();
    if (lane == 0) red[wave] = d;
    __syncthreads();
    if (tid == 0) {
      double x = 0.0;
      for (int w = 0; w < NW; ++w) x += red[w];
      J.xd_out[((long long)slab * a.segs + sid) * a.H + hd] = x;
    }
  }
}

// Contribution of one segment to the state behind it (before it, for a
// reversed job), written at that segment's place.  The last segment in the
// job's direction has none behind it and does nothing.
template <typename T, int DKP, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(LaTile<T, DKP, NW>::kWaves))) void
pdssm_linattn_state_kernel(const LaArgs a) {
  using K = LaTile<T, DKP, NW>;
  using E = typename T::store;
  using F = typename T::frag;
  constexpr int C = K::C;
  extern __shared__ __align__(16) unsigned char smem[];
  E* Y = (E*)smem;
  E* Z = (E*)(smem + K::kX);
  float* exps = (float*)(smem + K::kX + K::kZ);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5,
            n32 = lane & 31;
  unsigned id = blockIdx.x;
  const int jn = id % a.njobs;
  id /= a.njobs;
  const int slab = id % a.slabs;
  id /= a.slabs;
  const int hd = id % a.H;
  const int sid = id / a.H;
  const LaJob& J = a.job[jn];
  LaSeg s;
  if (!la_segment(a, sid, s)) return;
  const int rev = J.rev;
  if (rev ? s.first : s.last) return;
  const int slab0 = slab * NW * 32, c0 = slab0 + wave * 32, col = c0 + n32;
  const int chunks = (s.len + C - 1) / C;
  const E* yp = la_ptr<T>(J.y, s.vb, hd / J.yd, s.t0);
  const E* zp = la_ptr<T>(J.z, s.vb, hd / J.zd, s.t0) + slab0;
  const float* gp = (const float*)a.g.p + (int64_t)s.vb * a.g.sb + (int64_t)hd * a.g.sh + (int64_t)s.t0 * a.g.st;
  typename K::X ty;
  typename K::Z tz;
  ty.init(tid, J.DK);
  tz.init(tid, J.DV - slab0);
  float gv = 0.0f;
  constexpr int kExpWave = NW - 1;
  auto fetch = [&](int ci) {
    const int n = s.len - ci * C;
    ty.fetch(yp + (int64_t)(ci * C) * J.y.st, J.y.st, n);
    tz.fetch(zp + (int64_t)(ci * C) * J.z.st, J.z.st, n);
    if (wave == kExpWave) gv = lane < n && lane < C ? gp[(int64_t)(ci * C + lane) * a.g.st] : 0.0f;
  };
  if (chunks) fetch(rev ? chunks - 1 : 0);
  la_f16 S[K::KT];
#pragma unroll
  for (int t = 0; t < K::KT; ++t) S[t] = la_f16{};
  double sum = 0.0;
  if (wave == kExpWave) sum += la_exponents<C>(gv, rev, 1.0f, J.s_upd, exps, lane);
  for (int q = 0; q < chunks; ++q) {
    const int ci = rev ? chunks - 1 - q : q;
    const int n = s.len - ci * C < C ? s.len - ci * C : C;
    const float* e = exps + (q & 1) * K::kExp;
    ty.commit(Y, tid, n);
    tz.commit(Z, tid, n);
    __syncthreads();
    if (q + 1 < chunks) fetch(rev ? ci - 1 : ci + 1);
    F zf[C / 16];
#pragma unroll
    for (int js = 0; js < C / 16; ++js) zf[js] = T::col(Z, K::ZS, 16 * js, wave * 32, lane);
    la_update<T, DKP, NW>(S, Y, zf, e + 3 * C, e[4 * C], lane);
    if (wave == kExpWave && q + 1 < chunks)
      sum += la_exponents<C>(gv, rev, 1.0f, J.s_upd, exps + ((q + 1) & 1) * K::kExp, lane);
    __syncthreads();
  }
  const long long at = ((long long)(sid + (rev ? -1 : 1)) * a.H + hd);
  la_store_state<K::KT>(S, J.seg_out + at * a.state, J.sm, J.sn, J.DK, J.DV, col, h);
  if (slab == 0 && wave == kExpWave && lane == 0) J.seg_decay[at] = __builtin_amdgcn_exp2f((float)sum);
}

}  // namespace pdscan
