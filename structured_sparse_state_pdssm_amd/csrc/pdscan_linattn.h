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
// Exponents are differences of sums formed in 64 bits.  Where the decay over a
// chunk is moderate, a pair's weight is a factor of its query (2^A) times one of its
// key (2^-A, up to 2^24); else it is the power of the pair's own difference,
// at or below zero, of sums held as two floats, so a strong decay does not spoil
// the differences behind it.
//
// Precision.  bf16 inputs enter the products as they are.  What is computed
// (the state, the weighted scores, the weighted values) is held in fp32 and
// enters a product as two or three bf16 pieces, each the rest of those before
// it: two leave 2^-18 of a term (enough for outputs that are rounded to bf16,
// at 2^-9), three nothing (states and what the log-decay gradient is summed
// from).  fp32 inputs are three pieces themselves.
#pragma once

#include <hip/hip_runtime.h>

#include "pdscan_linattn_plan.h"

namespace pdscan {

typedef __bf16 la_bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 la_bf2 __attribute__((ext_vector_type(2)));
typedef float la_f2 __attribute__((ext_vector_type(2)));
typedef float la_f16 __attribute__((ext_vector_type(16)));
typedef short la_s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) la_s4 la_lds_s4;

// ---- operand layout
//
// A 32 x 32 x 16 product takes from lane (n = lane % 32, h = lane / 32) the
// eight contraction slots of its half and leaves in accumulator register r
// the row 8 (r / 4) + 4 h + r % 4 of column n.  Rows are fed in the order
// pi(m) = m with bits 2 and 3 exchanged, so registers 8 s .. 8 s + 7 of a lane
// hold the rows 16 s + 8 h .. + 7: eight neighbours.  They are stored and read
// 16 bytes at a time, and they are exactly the slots that the next product's
// operand wants of that lane, so an accumulator becomes an operand without any
// exchange between lanes.
__device__ __forceinline__ int la_pi(int m) { return (m & ~12) | ((m & 4) << 1) | ((m & 8) >> 1); }

// ---- LDS layout
//
// Tiles lie row by row without padding; 16-byte unit u of row r is kept at
// unit u ^ f(r).  f is linear in the bits of r and such that 16 rows read at
// one unit (row operands), and four rows read at four neighbouring units
// (column operands through the transposing read), fall on different banks.
template <int ROW_BYTES>
__device__ __forceinline__ constexpr int la_f(int r) {
  return ROW_BYTES >= 256   ? ((((r & 3) << 2) | ((r >> 2) & 3)) ^ (r & 8))
         : ROW_BYTES == 128 ? (((r >> 1 & 1) << 2) | (r >> 2 & 3))
                            : (r >> 2 & 3);
}

struct LaBf16 {
  using store = uint16_t;
  static constexpr int kVec = 8;    // elements of 16 bytes
  static constexpr int kPlanes = 1; // bf16 values that an element is in LDS
  union frag {
    uint32_t u[4];
    uint4 w;
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
  static __device__ __forceinline__ void unpack(const uint4* p, float* v) {   // eight elements
    const uint32_t u[4] = {p->x, p->y, p->z, p->w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  }
  // eight elements of a row at byte address a (PS: bytes of a plane)
  template <int PS>
  static __device__ __forceinline__ frag row(const unsigned char* a) {
    frag f;
    f.w = *(const uint4*)a;
    return f;
  }
  // Byte offset, for this lane, of column operands: rows 8 h .. 8 h + 7 of the
  // columns pi(0 .. 31).  The transposing read hands the 16 lanes of a group
  // four rows of four times four columns: lane p points at row p / 4, its
  // (p % 4)-th four columns, and receives column p; pi swaps the second and
  // third four.
  template <int RB>
  static __device__ __forceinline__ uint32_t col_base(int lane, int c0) {
    const int p = lane & 15, r = 8 * (lane >> 5) + (p >> 2), q = p & 3, c4 = ((q & 1) << 1) | (q >> 1);
    const int unit = c0 / 8 + ((lane & 16) >> 3) + (c4 >> 1);
    return r * RB + ((unit ^ la_f<RB>(r)) << 4) + (c4 & 1) * 8;
  }
  template <int RB, int PS>
  static __device__ __forceinline__ frag col(const unsigned char* lds, uint32_t base, int r0, int tile) {
    const uint32_t b = base ^ (uint32_t)(tile * 64);
    frag f;
    f.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((la_lds_s4*)(lds + b + r0 * RB));
    f.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((la_lds_s4*)(lds + (b ^ (la_f<RB>(4) << 4)) + (r0 + 4) * RB));
    return f;
  }
  static __device__ __forceinline__ uint32_t round2(float x, float y) {   // nearest, ties to even
    const la_f2 v = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, la_bf2));
  }
  // two floats rounded to bf16, and what is left of them (exactly)
  static __device__ __forceinline__ uint32_t split2(float& x, float& y) {
    const uint32_t w = round2(x, y);
    x -= __uint_as_float(w << 16);
    y -= __uint_as_float(w & 0xffff0000u);
    return w;
  }
  // eight floats as bf16 pieces, each the rest of those before rounded to the
  // nearest: two leave 2^-18 of a value, three nothing.  (Cut pieces cost the
  // same, leave 2^-16 and all on one side, which adds up over long sums.)
  template <int NP>
  static __device__ __forceinline__ void pieces(const float* v, frag* out) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = v[2 * e], y = v[2 * e + 1];
#pragma unroll
      for (int p = 0; p + 1 < NP; ++p) out[p].u[e] = split2(x, y);
      out[NP - 1].u[e] = round2(x, y);
    }
  }
  static __device__ __forceinline__ void put(unsigned char* a, const frag& f) { *(uint4*)a = f.w; }
  // 16 bytes of a row from memory to their place, column c in it, of a row of RB bytes (XOR x from its swizzle)
  template <int RB, int PS>
  static __device__ __forceinline__ void put_row(unsigned char* lds, int row, int c, uint32_t x, const uint4& w) {
    *(uint4*)(lds + ((row * RB + (((c >> 3) ^ la_f<RB>(row)) << 4)) ^ x)) = w;
  }
  static __device__ __forceinline__ void store4(store* p, const float* v) {
    *(uint2*)p = make_uint2(round2(v[0], v[1]), round2(v[2], v[3]));
  }
  static __device__ __forceinline__ void store8(store* p, const float* v) {
    *(uint4*)p = make_uint4(round2(v[0], v[1]), round2(v[2], v[3]), round2(v[4], v[5]), round2(v[6], v[7]));
  }
  static __device__ __forceinline__ void load4(const store* p, float* v) {
    const uint2 w = *(const uint2*)p;
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
};

// fp32 elements are three bf16 pieces in LDS, a plane each, whose sum is the
// element; of the nine products of two elements the six of weight 2^-18 and up
// are formed, which leaves 2^-26 of a term.  Six bf16 products take 3/8 of the
// time of the fp32 ones.
struct LaF32 {
  using store = float;
  static constexpr int kVec = 4;
  static constexpr int kPlanes = 3;
  struct frag {
    LaBf16::frag p[3];
  };
  static __device__ __forceinline__ void mma(la_f16& c, const frag& a, const frag& b) {
    LaBf16::mma(c, a.p[0], b.p[2]);
    LaBf16::mma(c, a.p[2], b.p[0]);
    LaBf16::mma(c, a.p[1], b.p[1]);
    LaBf16::mma(c, a.p[0], b.p[1]);
    LaBf16::mma(c, a.p[1], b.p[0]);
    LaBf16::mma(c, a.p[0], b.p[0]);
  }
  static __device__ __forceinline__ float get(const frag& f, int e) {
    return (LaBf16::get(f.p[0], e) + LaBf16::get(f.p[1], e)) + LaBf16::get(f.p[2], e);
  }
  static __device__ __forceinline__ void unpack(const uint4* p, float* v) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      v[4 * u] = __uint_as_float(p[u].x);
      v[4 * u + 1] = __uint_as_float(p[u].y);
      v[4 * u + 2] = __uint_as_float(p[u].z);
      v[4 * u + 3] = __uint_as_float(p[u].w);
    }
  }
  template <int PS>
  static __device__ __forceinline__ frag row(const unsigned char* a) {
    frag f;
#pragma unroll
    for (int p = 0; p < 3; ++p) f.p[p] = LaBf16::row<0>(a + p * PS);
    return f;
  }
  template <int RB>
  static __device__ __forceinline__ uint32_t col_base(int lane, int c0) {
    return LaBf16::col_base<RB>(lane, c0);
  }
  template <int RB, int PS>
  static __device__ __forceinline__ frag col(const unsigned char* lds, uint32_t base, int r0, int tile) {
    frag f;
#pragma unroll
    for (int p = 0; p < 3; ++p) f.p[p] = LaBf16::col<RB, 0>(lds + p * PS, base, r0, tile);
    return f;
  }
  template <int NP>
  static __device__ __forceinline__ void pieces(const float* v, frag* out) {
    LaBf16::pieces<3>(v, out[0].p);
  }
  template <int RB, int PS>
  static __device__ __forceinline__ void put_row(unsigned char* lds, int row, int c, uint32_t x, const uint4& w) {
    unsigned char* a = lds + ((row * RB + (((c >> 3) ^ la_f<RB>(row)) << 4) + (c & 4) * 2) ^ x);
    float v[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const uint32_t lo = LaBf16::split2(v[0], v[1]), hi = LaBf16::split2(v[2], v[3]);
      *(uint2*)(a + p * PS) = make_uint2(lo, hi);
    }
  }
  static __device__ __forceinline__ void store4(store* p, const float* v) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  }
  static __device__ __forceinline__ void store8(store* p, const float* v) {
    store4(p, v);
    store4(p + 4, v + 4);
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

// This workgroup's number in a grid of la_grid_rows, `row` of them along x.
__device__ __forceinline__ unsigned la_block(unsigned row) { return blockIdx.y * row + blockIdx.x; }

struct LaUnit {
  int job, slab, hd, sid;
};

// What workgroup `id` works on: those that share rows follow one another.
__device__ __forceinline__ void la_unit(const LaArgs& a, unsigned id, LaUnit& u) {
  u.job = id % a.njobs;
  id /= a.njobs;
  u.slab = id % a.slabs;
  id /= a.slabs;
  u.hd = id % a.H;
  u.sid = id / a.H;
}

template <typename T>
__device__ __forceinline__ const typename T::store* la_ptr(const LaView& v, int b, int h, int t) {
  return (const typename T::store*)v.p + (int64_t)b * v.sb + (int64_t)h * v.sh + (int64_t)t * v.st;
}

// A tile of C rows and W elements on its way from memory to LDS: thread
// `tid` owns 16 bytes of every RP-th row.  fetch() only issues the loads (the
// next chunk's while this one is worked on); rows behind n and columns behind
// D are loaded from a place that exists and become zero in commit().  The
// chunk's place is uniform, a lane adds 32 bits (the host bounds the stride).
template <typename T, int C, int W, int NT>
struct LaTileIO {
  using E = typename T::store;
  static constexpr int kCols = W / T::kVec, RP = NT / kCols, N = C / RP, RB = W * 2, PS = C * RB;
  static_assert(RP * kCols == NT && N * RP == C, "whole passes");
  uint4 r[N];
  const char* base;      // the chunk under way
  uint32_t st, off;      // bytes of a row's stride; this thread's offset
  int row0;
  bool ok;
  __device__ __forceinline__ void init(const E* chunk, int64_t stride, int tid, int D) {
    base = (const char*)chunk;
    st = (uint32_t)stride * (uint32_t)sizeof(E);
    row0 = tid / kCols;
    const int col = tid % kCols * T::kVec;
    ok = col < D;
    off = row0 * st + (ok ? col : 0) * (uint32_t)sizeof(E);
  }
  __device__ __forceinline__ void fetch(int n) {
    if (n >= C) {
      uint32_t o = off;
#pragma unroll
      for (int i = 0; i < N; ++i, o += RP * st) r[i] = *(const uint4*)(base + o);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = row0 + i * RP;
        r[i] = *(const uint4*)(base + (uint32_t)(off + (uint32_t)((row < n ? row : n - 1) - row0) * st));
      }
    }
  }
  __device__ __forceinline__ void commit(unsigned char* lds, int tid, int n, bool whole) {
    if (!whole) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!ok || row0 + i * RP >= n) r[i] = make_uint4(0, 0, 0, 0);
    }
    const int c = tid % kCols * T::kVec;
#pragma unroll
    for (int i = 0; i < N; ++i)
      T::template put_row<RB, PS>(lds + i * RP * RB, row0, c, (uint32_t)(la_f<RB>(i * RP) << 4), r[i]);
  }
};

// x plus the value of the lane that DPP control CTRL names (zero where there
// is none or the row is masked)
template <int CTRL, int ROWS>
__device__ __forceinline__ double la_scan_step(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return x + __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// 2^x, x in 64 bits: whole part and rest apart, so that large |x| costs no digits.
__device__ __forceinline__ float la_exp2(double x) {
  const double n = __builtin_rint(x);
  const float f = __builtin_amdgcn_exp2f((float)(x - n));
  return __builtin_amdgcn_ldexpf(f, x < -1000.0 ? -1000 : (int)n);
}

// Inclusive sums of log2 decay over each of 64 / C chunks (lane = token, chunk
// by chunk in the job's direction; g = its log decay, 0 behind the last), and
// at `l` lane l's.  A log decay under -1e4 (minus infinity: the state starts
// anew) counts as -1e4, whose exponential is zero all the same.
template <int C>
__device__ __forceinline__ double la_scan(float g) {
  if (g < -1e4f) g = -1e4f;
  double G = (double)g * 1.4426950408889634074;
  G = la_scan_step<0x111, 0xf>(G);   // row_shr:1
  G = la_scan_step<0x112, 0xf>(G);   // row_shr:2
  G = la_scan_step<0x114, 0xf>(G);   // row_shr:4
  G = la_scan_step<0x118, 0xf>(G);   // row_shr:8
  G = la_scan_step<0x142, 0xa>(G);   // row_bcast:15 into rows 1 and 3
  if constexpr (C == 64) G = la_scan_step<0x143, 0xc>(G);   // row_bcast:31 into rows 2 and 3
  return G;
}
__device__ __forceinline__ double la_lane(double x, int l) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// What the tokens of 64 / C chunks are weighted with in the product kernel, by
// one wave (lanes as in la_scan).  With A the log2 of the decay between a token and its chunk's entering state
// (G, or G_C - G backwards), e, kExp floats per chunk, gets
//   e[2C + i] = 2^A s_out, the output's scale
//   e[3C + j] the update's weight
//   e[4C]     the chunk's whole decay
//   e[4C + 1] 1 where no |A| is above kLaNear: then the weight of a pair is
//             2^{A_i} 2^{-A_j}, its first factor common to the whole output,
//             and e[j] = 2^{-A_j} s_ratio; else 0, and e[i], e[C + i] hold G as
//             two floats for the difference of every pair.
template <int C, int EXP>
__device__ __forceinline__ void la_exponents(float g, int rev, float s_out, float s_ratio, float s_upd, float* e,
                                             int lane) {
  const double G = la_scan<C>(g);
  double tot = la_lane(G, 63);
  if (C == 32 && lane < 32) tot = la_lane(G, 31);
  const double A = rev ? tot - G : G, B = rev ? G : tot - G;
  const uint64_t far_lanes = __ballot(!(A <= kLaNear && A >= -kLaNear));
  const bool near = C == 64 ? far_lanes == 0 : (lane < 32 ? (uint32_t)far_lanes : (uint32_t)(far_lanes >> 32)) == 0;
  const int i = lane & (C - 1);
  e += C == 64 ? 0 : (lane >> 5) * EXP;
  if (near) {
    e[i] = la_exp2(-A) * s_ratio;
  } else {
    const float gh = (float)G;
    e[i] = gh;
    e[C + i] = (float)(G - (double)gh);
  }
  e[2 * C + i] = la_exp2(A) * s_out;
  e[3 * C + i] = la_exp2(B) * s_upd;
  if (i == 0) {
    e[4 * C] = la_exp2(tot);
    e[4 * C + 1] = near ? 1.0f : 0.0f;
  }
}

template <typename T, int DKP, int NW>
struct LaTile {
  static constexpr bool kF32 = sizeof(typename T::store) == 4;
  static constexpr int C = la_chunk(NW, !kF32);  // tokens of a chunk
  static constexpr int NT = NW * 64;
  static constexpr int IT = C / 32;              // 32-token tiles of a chunk
  static constexpr int KT = DKP / 32;            // 32-row tiles of the state
  static constexpr int WV = kF32 ? 2 : 1;        // 16-byte units of eight elements
  static constexpr int NPS = kF32 ? 1 : 3;       // pieces of the state's update
  // One or two waves form all scores of the chunk each, in registers, and so do
  // four in fp32; four in bf16 share them through LDS (a tile of 32 x 32 each).
  static constexpr bool kShareP = NW == 4 && !kF32;
  static constexpr int ES = (int)sizeof(typename T::store);
  static constexpr int XB = DKP * 2, ZB = NW * 64, PB = C * 2;   // bytes of a row in LDS
  static constexpr int XP = C * XB, ZP = C * ZB;                 // and of a plane
  static constexpr int kExp = 4 * C + 4;         // floats of one chunk's exponents
  static constexpr size_t kX = (size_t)T::kPlanes * XP, kZ = (size_t)T::kPlanes * ZP, kP = kShareP ? (size_t)C * PB : 0;
  static constexpr int PAIR = 64 / C;            // chunks whose exponents are formed at once
  static constexpr size_t kSmall = (size_t)(2 * PAIR * kExp + (NW + 1) * C) * 4;
  static constexpr int pieces(int mode) { return kF32 ? 1 : mode == kLaQ || mode == kLaK ? 3 : 2; }
  static constexpr size_t main_bytes(int np) { return 2 * kX + kZ + np * kP + kSmall; }
  static_assert(main_bytes(2) == (size_t)la_lds(DKP, NW, !kF32, 2) && main_bytes(3) == (size_t)la_lds(DKP, NW, !kF32, 3),
                "what the plan counts");
  static constexpr size_t state_bytes() { return 2 * (kX + kZ) + (size_t)NW * 64 * 4; }
  using X = LaTileIO<T, C, DKP, NT>;
  using Z = LaTileIO<T, C, NW * 32, NT>;
  // rows of 256 elements: the scheduler is kept from loading more operands ahead than the registers hold
  static constexpr bool kWide = KT == 8;
  static constexpr bool kApart = kF32 || KT < 4 || (KT == 4 && !kShareP);
  static constexpr int kWaves = la_simd_waves(la_regs(KT + IT, 2 * X::N + Z::N, kF32));
  // The state kernel's, by the same count of its own registers in fp32.  Forward passes: 65536 steps, 4 heads, 128/32
  // (174) 214 us instead of 235 at two, where it spills 30; 2 x 2048 steps, 8 heads, 256/256 (194) 174 instead of
  // 232.  bf16 stays at two: rows of 256 with four waves spill 2 there and take the same (4 x 2048 steps, 12 heads,
  // 256/256 208 us either way, its gradient 640 against 645).
  static constexpr int kStateWaves = kF32 ? la_simd_waves(la_regs(KT, X::N + Z::N, true)) : 2;
};

// S = decay S + sum_j y_j (w_j z_j)^T (KEEP: S as it is).  A matrix instruction
// adds eight of its 16 products to the accumulator at a time, rounded to the
// nearest (ties to even), so a term in three pieces costs the state twelve roundings for
// 32 tokens, one in fp32 24.  Formed apart, their sum costs it one.  Over 8192
// same-signed steps without decay: 2.3e-7 off apart, 4.5e-7 in place, and the mean
// error under 3e-8 either way.  In place where the registers do not hold the
// sum (APART false): bf16 rows of 128 elements with four waves, 311 us instead of
// 175 for a gradient, and of 256.
template <typename T, int DKP, int NW, bool KEEP, bool APART>
__device__ __forceinline__ void la_update(la_f16 (&S)[DKP / 32], const unsigned char* Y, uint32_t ycol,
                                          const typename T::frag* zf, const float* ew, float decay, int lane) {
  using K = LaTile<T, DKP, NW>;
  const int h = lane >> 5;
  if constexpr (!KEEP && !APART) {
#pragma unroll
    for (int t = 0; t < K::KT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[t][r] *= decay;
  }
#pragma unroll
  for (int g = 0; g < K::C / 32; ++g) {
    typename T::frag b[2][K::NPS];
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      const int js = 2 * g + k2;
      float v[8];
      const float4 w0 = *(const float4*)(ew + 16 * js + 8 * h), w1 = *(const float4*)(ew + 16 * js + 8 * h + 4);
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = T::get(zf[js], e) * w[e];
      T::template pieces<K::NPS>(v, b[k2]);
      if constexpr (!APART) {
#pragma unroll
        for (int t = 0; t < K::KT; ++t) {
          const typename T::frag y = T::template col<K::XB, K::XP>(Y, ycol, 16 * js, t);
#pragma unroll
          for (int p = 0; p < K::NPS; ++p) T::mma(S[t], y, b[k2][K::NPS - 1 - p]);
          if (K::kWide) __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    if constexpr (!APART) continue;
#pragma unroll
    for (int t = 0; t < K::KT; ++t) {
      la_f16 d = {};
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        const typename T::frag y = T::template col<K::XB, K::XP>(Y, ycol, 16 * (2 * g + k2), t);
#pragma unroll
        for (int p = 0; p < K::NPS; ++p) T::mma(d, y, b[k2][K::NPS - 1 - p]);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) S[t][r] = KEEP || g > 0 ? S[t][r] + d[r] : __builtin_fmaf(S[t][r], decay, d[r]);
      if (K::kWide) __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// A state's rows m and column `col` of this lane, zero where p is NULL or the
// state ends.  sm = 1: the rows lie side by side (the state is stored
// transposed) and come four to a load.
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
    for (int s = 0; s < 2; ++s) {
      const int m = 32 * t + 16 * s + 8 * h;
      const bool in = m < DK && col < DV;
      const int mm = m < DK ? m : 0;
      float v[8];
      if (sm == 1) {
        *(float4*)&v[0] = *(const float4*)(q + mm);
        *(float4*)&v[4] = *(const float4*)(q + mm + 4);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = q[(long long)(mm + e) * sm];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) S[t][8 * s + e] = in ? v[e] : 0.0f;
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
    for (int s = 0; s < 2; ++s) {
      const int m = 32 * t + 16 * s + 8 * h;
      if (m >= DK) continue;
      if (sm == 1) {
        *(float4*)(q + m) = make_float4(S[t][8 * s], S[t][8 * s + 1], S[t][8 * s + 2], S[t][8 * s + 3]);
        *(float4*)(q + m + 4) = make_float4(S[t][8 * s + 4], S[t][8 * s + 5], S[t][8 * s + 6], S[t][8 * s + 7]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[(long long)(m + e) * sm] = S[t][8 * s + e];
      }
    }
}

// Scores of one 32 x 32 tile (rows j of y, columns i of x), weighted by the
// decay between the two tokens (near: by the part of it that is the key's) and
// zero on the wrong side of the diagonal.  DIAG: zero on it too, and d is the
// diagonal's element of column i (zero in the half of the lanes without it).
template <typename T, int DKP, int NW, bool REV, bool DIAG>
__device__ __forceinline__ la_f16 la_scores(const unsigned char* X, const unsigned char* Y, uint32_t xrow,
                                            uint32_t yrow, const float* e, bool near, int jt, int it, float s_intra,
                                            int lane, float& d) {
  using K = LaTile<T, DKP, NW>;
  const int h = lane >> 5, n32 = lane & 31;
  la_f16 c = {};
#pragma unroll
  for (int ks = 0; ks < DKP / 16; ++ks) {
    T::mma(c, T::template row<K::XP>(Y + (yrow ^ (uint32_t)(ks * 32)) + jt * 32 * K::XB),
           T::template row<K::XP>(X + (xrow ^ (uint32_t)(ks * 32)) + it * 32 * K::XB));
    if (K::kWide && ks % 2) __builtin_amdgcn_sched_barrier(0);
  }
  const int j0 = 32 * jt + 8 * h;
  if (near) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float w[8];
      *(float4*)&w[0] = *(const float4*)(e + j0 + 16 * s);
      *(float4*)&w[4] = *(const float4*)(e + j0 + 16 * s + 4);
#pragma unroll
      for (int q = 0; q < 8; ++q) c[8 * s + q] *= w[q];
    }
  } else {
    const int i = 32 * it + n32;
    const float gi = e[i], gl = e[K::C + i];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float hh[8], ll[8];
      *(float4*)&hh[0] = *(const float4*)(e + j0 + 16 * s);
      *(float4*)&hh[4] = *(const float4*)(e + j0 + 16 * s + 4);
      *(float4*)&ll[0] = *(const float4*)(e + K::C + j0 + 16 * s);
      *(float4*)&ll[4] = *(const float4*)(e + K::C + j0 + 16 * s + 4);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float x = REV ? (hh[q] - gi) + (ll[q] - gl) : (gi - hh[q]) + (gl - ll[q]);
        c[8 * s + q] *= __builtin_amdgcn_exp2f(x) * s_intra;
      }
    }
  }
  if (jt == it) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int j = 16 * s + 8 * h + q;
        if (DIAG && j == n32) d = c[8 * s + q];
        if (REV ? DIAG ? j <= n32 : j < n32 : DIAG ? j >= n32 : j > n32) c[8 * s + q] = 0.0f;
      }
  }
  return c;
}

// o = form(x, y, z) over one segment, head and slab of 32 NW columns.
// MODE: the forward pass, or one of the gradient's jobs.  Those of q and k
// also give w . o per token (for the log-decay gradient, so with three pieces
// throughout); that of q multiplies the final state with its gradient.
//
// A chunk's tiles are loaded once, a chunk ahead, and everything but o stays in
// registers and LDS, so few rows of input are waited for at once and the work
// of a chunk is a chain: scores, their pieces, the products, the state.  In most
// sizes memory bounds it: whole 128-byte lines move behind the L2s, more than once where
// heads that share them run on several dies (a large copy has 4.7 TB/s, reads and writes;
// what is above comes from the cache there).  With three pieces of 128-wide rows it is that chain.
//   forward  16 x 2048, 24 heads, 64/32 bf16    70 us, 396 MB at 5.6 TB/s (matrix 9, VALU 19, LDS 8)
//            65536 steps, 16 heads, 128/128    264 us, 1145 MB at 4.3 (matrix 84, VALU 77, LDS 47)
//            4 x 4096, 8 heads, 16/64 fp32      25 us, 105 MB at 4.1 (matrix 5, VALU 10, LDS 3)
//   dq and dk of the first of these            209 us, 1067 MB at 5.1 (matrix 26, VALU 94, LDS 22), dv 70 us
//   dq, dk, dv of 8190 rows, 16 heads, 128/128 179 us, 627 MB at 3.5 (matrix 38, VALU 45, LDS 21)
// (matrix, VALU, LDS: the time that those alone take of a SIMD or an LDS.)  A call
// of few steps is its start-up: 5 to 7 us, and 2 to 6 for a chunk of 32 (64/64).
template <typename T, int DKP, int NW, int MODE>
__device__ __forceinline__ void la_body(const LaArgs& a, const LaJob& J, const LaSeg& s, int sid, int hd, int slab,
                                        unsigned char* smem) {
  using K = LaTile<T, DKP, NW>;
  using E = typename T::store;
  using F = typename T::frag;
  constexpr int C = K::C, IT = K::IT, NP = K::pieces(MODE);
  constexpr bool REV = MODE == kLaK || MODE == kLaV, dot = MODE == kLaQ || MODE == kLaK;
  unsigned char* X = smem;
  unsigned char* Y = smem + K::kX;
  unsigned char* Z = smem + 2 * K::kX;
  unsigned char* P = smem + 2 * K::kX + K::kZ;
  float* exps = (float*)(smem + 2 * K::kX + K::kZ + NP * K::kP);   // of the chunks under way and the next
  float* dots = exps + 2 * K::PAIR * K::kExp;                      // [NW][C]
  float* diag = dots + NW * C;                                     // [C]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5,
            n32 = lane & 31, pm = la_pi(n32);
  const int slab0 = slab * NW * 32;
  const int c0 = slab0 + wave * 32;      // first column of this wave
  const int col = c0 + pm;               // the state's column of this lane
  const long long unit = (long long)s.b * a.H + hd;
  const int chunks = (s.len + C - 1) / C;
  const int first = REV ? (chunks ? chunks - 1 : 0) * C : 0;   // first step worked on
  constexpr int dir = REV ? -C : C;
  typename K::X tx, ty;
  typename K::Z tz;
  tx.init(la_ptr<T>(J.x, s.vb, hd / J.xd, s.t0 + first), J.x.st, tid, J.DK);
  ty.init(la_ptr<T>(J.y, s.vb, hd / J.yd, s.t0 + first), J.y.st, tid, J.DK);
  tz.init(la_ptr<T>(J.z, s.vb, hd / J.zd, s.t0 + first) + slab0, J.z.st, tid, J.DV - slab0);
  const int64_t dx = dir * J.x.st * K::ES, dy = dir * J.y.st * K::ES, dz = dir * J.z.st * K::ES, dg = dir * a.g.st;
  const bool whole = J.DK == DKP && J.DV - slab0 >= NW * 32;
  const float* gp = (const float*)a.g.p + (int64_t)s.vb * a.g.sb + (int64_t)hd * a.g.sh +
                    (int64_t)(s.t0 + first) * a.g.st;
  const int64_t goff = (lane & (C - 1)) * a.g.st + (lane / C) * dg;
  constexpr int PAIR = K::PAIR;
  // The wave that forms the weights: with shared scores the one whose tile
  // lies on the wrong side of the diagonal, while the others work on theirs.
  constexpr int kExpWave = K::kShareP && IT == 2 ? (REV ? 1 : 2) : NW - 1;
  auto fetch = [&](int n) {
    tx.fetch(n);
    ty.fetch(n);
    tz.fetch(n);
  };
  // log decays of PAIR chunks, the first of them `skip` chunks on from step `at`
  auto fetch_g = [&](int at, int skip) {
    const int mine = skip + lane / C;
    const int n = REV ? (at >= mine * C ? s.len - (at - mine * C) : 0) : s.len - at - mine * C;
    float g = 0.0f;
    if (wave == kExpWave && (lane & (C - 1)) < n) g = gp[goff + skip * dg];
    return g;
  };
  float gv = 0.0f, g0 = 0.0f;
  if (chunks) {
    g0 = fetch_g(first, 0);
    if (PAIR == 1) gv = fetch_g(first, 1);
    fetch(s.len - first);
  }

  la_f16 S[K::KT];
  {
    const bool starts = REV ? s.last : s.first;
    const float* init = starts ? (J.s_user ? J.s_user + unit * a.state : nullptr)
                               : J.s_seg + ((long long)sid * a.H + hd) * a.state;
    la_load_state<K::KT>(S, init, J.sm, J.sn, J.DK, J.DV, col, h);
  }
  if (wave == kExpWave) la_exponents<C, K::kExp>(g0, REV, J.s_out, J.s_ratio, J.s_upd, exps, lane);

  // lane offsets of the operands in LDS
  uint32_t xrow = n32 * K::XB + ((h ^ la_f<K::XB>(n32)) << 4);
  uint32_t yrow = pm * K::XB + ((h ^ la_f<K::XB>(pm)) << 4);
  uint32_t ycol = T::template col_base<K::XB>(lane, 0);
  uint32_t zcol = T::template col_base<K::ZB>(lane, wave * 32);
  uint32_t zrow = n32 * K::ZB + (((wave * 4 + h) ^ la_f<K::ZB>(n32)) << 4);
  uint32_t prow = n32 * K::PB + ((h ^ la_f<K::PB>(n32)) << 4);

  const int oes = dot && J.o_f32 ? 4 : K::ES;
  char* ob = (char*)J.o.p +
             ((int64_t)s.vb * J.o.sb + (int64_t)(hd / J.od) * J.o.sh + (int64_t)(s.t0 + first) * J.o.st + c0) * oes;
  const uint32_t ost = (uint32_t)J.o.st * (uint32_t)oes, ooff = n32 * ost + 8 * h * oes;
  const char* wb = nullptr;
  uint32_t wst = 0, woff = 0;
  if (dot) {
    wb = (const char*)(la_ptr<T>(J.w, s.vb, hd / J.wd, s.t0 + first) + c0);
    wst = (uint32_t)J.w.st * K::ES;
    woff = n32 * wst + 8 * h * K::ES;
  }
  const float s_out = J.s_out, s_ratio = J.s_ratio, s_upd = J.s_upd, s_intra = s_out * s_ratio;
  int n = s.len - first;                 // steps of this chunk
  int at = first;                        // its first step in the segment

  for (int q = 0; q < chunks; ++q) {
    if (n > C) n = C;
    // the operands' places are one exclusive-or away from these: cheaper than the registers to keep them all
    asm volatile("" : "+v"(xrow), "+v"(yrow), "+v"(ycol), "+v"(zcol), "+v"(zrow), "+v"(prow));
    const float* e = exps + (q % (2 * PAIR)) * K::kExp;
    tx.commit(X, tid, n, whole && n == C);
    ty.commit(Y, tid, n, whole && n == C);
    tz.commit(Z, tid, n, whole && n == C);
    __syncthreads();
    // loads are waited for in order: w, which this chunk needs, before the next chunk's tiles
    uint4 wv[IT][2 * K::WV];
    if (dot) {
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int i = 32 * it + n32;
        const char* wp = wb + (uint32_t)(woff + (uint32_t)((i < n ? i : n - 1) - n32) * wst);
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
          for (int u = 0; u < K::WV; ++u)
            wv[it][k2 * K::WV + u] =
                *(const uint4*)(wp + (c0 + 16 * k2 + 8 * h < J.DV ? 16 * k2 * K::ES + 16 * u : -(c0 + 8 * h) * K::ES));
      }
    }
    // the log decays two chunks on: their weights are formed in the next chunk's time
    const float gnext = q % PAIR == 0 ? fetch_g(at, 2) : gv;
    if (q + 1 < chunks) {
      tx.base += dx;
      ty.base += dy;
      tz.base += dz;
      gp += dg;
      fetch(REV ? C : s.len - at - C);
    }
    const bool near = __builtin_amdgcn_readfirstlane(__float_as_int(e[4 * C + 1])) != 0;
    if constexpr (K::kShareP) {
      static_assert(IT * IT <= NW, "a score tile per wave");
      if (wave == kExpWave && q + 1 < chunks && q % PAIR == PAIR - 1)
        la_exponents<C, K::kExp>(gv, REV, s_out, s_ratio, s_upd, exps + ((q + 1) % (2 * PAIR)) * K::kExp, lane);
      const int jt = wave / IT, it = wave % IT;
      if (wave < IT * IT && (REV ? jt >= it : jt <= it)) {
        float d = 0.0f;
        const la_f16 c = la_scores<T, DKP, NW, REV, dot>(X, Y, xrow, yrow, e, near, jt, it, s_intra, lane, d);
        if (dot && jt == it) {
          d += __shfl_xor(d, 32, 64);
          if (h == 0) diag[32 * it + n32] = d;
        }
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
          float v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] = c[8 * k2 + r];
          F pp[NP];
          T::template pieces<NP>(v, pp);
#pragma unroll
          for (int p = 0; p < NP; ++p)
            T::put(P + p * K::kP + (prow ^ (uint32_t)((2 * jt + k2) * 32)) + it * 32 * K::PB, pp[p]);
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
          const F xb = T::template row<K::XP>(X + (xrow ^ (uint32_t)((2 * t4 + k2) * 32)) + it * 32 * K::XB);
#pragma unroll
          for (int p = 0; p < NP; ++p) T::mma(o[it], sp[p], xb);
        }
        if (K::kWide) __builtin_amdgcn_sched_barrier(0);
      }
    auto scale_out = [&]() {
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const float w = e[2 * C + 32 * it + n32];
#pragma unroll
        for (int r = 0; r < 16; ++r) o[it][r] *= w;
      }
    };
    if (!near) scale_out();   // near: the chunk's own part has the same factor

    // what the chunk's own tokens give
    F zf[C / 16];
#pragma unroll
    for (int js = 0; js < C / 16; ++js) zf[js] = T::template col<K::ZB, K::ZP>(Z, zcol, 16 * js, 0);
    float dv[IT];   // the token's own score, left out of the product where w . o is asked for
    if constexpr (K::kShareP) {
      __syncthreads();
      if (dot)
#pragma unroll
        for (int it = 0; it < IT; ++it) dv[it] = diag[32 * it + n32];
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int js = 0; js < C / 16; ++js) {
          if (REV ? js < 2 * it : js >= 2 * it + 2) continue;
#pragma unroll
          for (int p = 0; p < NP; ++p)
            T::mma(o[it], zf[js], T::template row<0>(P + p * K::kP + (prow ^ (uint32_t)(js * 32)) + it * 32 * K::PB));
        }
    } else {
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int jt = 0; jt < IT; ++jt) {
          if (REV ? jt < it : jt > it) continue;
          __builtin_amdgcn_sched_barrier(0);   // one tile at a time: all at once would not fit the registers
          float d = 0.0f;
          const la_f16 c = la_scores<T, DKP, NW, REV, dot>(X, Y, xrow, yrow, e, near, jt, it, s_intra, lane, d);
          if (dot && jt == it) dv[it] = d + __shfl_xor(d, 32, 64);
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

    if (near) scale_out();

#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int i = 32 * it + n32;
      float dsum = 0.0f, own = 0.0f;
      if (dot) own = near ? dv[it] * e[2 * C + i] : dv[it];
      char* oi = ob + (ooff + 32 * it * ost);
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        float v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = o[it][8 * k2 + r];
        if (dot) {
          // w . o without the token's own part: it is the same in the jobs of
          // q and k and cancels in their difference, but for rounding
          float w[8];
          T::unpack(&wv[it][k2 * K::WV], w);
          if (c0 + 16 * k2 + 8 * h < J.DV)
            dsum += ((w[0] * v[0] + w[1] * v[1]) + (w[2] * v[2] + w[3] * v[3])) +
                    ((w[4] * v[4] + w[5] * v[5]) + (w[6] * v[6] + w[7] * v[7]));
          const F z = T::template row<K::ZP>(Z + (zrow ^ (uint32_t)(k2 * 32)) + it * 32 * K::ZB);
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] += own * T::get(z, r);
        }
        if (i < n && c0 + 16 * k2 + 8 * h < J.DV) {
          if (dot && J.o_f32)
            LaF32::store8((float*)oi + 16 * k2, v);
          else
            T::store8((E*)oi + 16 * k2, v);
        }
      }
      if (dot) {
        dsum += __shfl_xor(dsum, 32, 64);
        if (h == 0) dots[wave * C + i] = dsum;
      }
    }

    __builtin_amdgcn_sched_barrier(0);
    la_update<T, DKP, NW, false, K::kApart>(S, Y, ycol, zf, e + 3 * C, e[4 * C], lane);
    if (!K::kShareP && wave == kExpWave && q + 1 < chunks && q % PAIR == PAIR - 1)
      la_exponents<C, K::kExp>(gv, REV, s_out, s_ratio, s_upd, exps + ((q + 1) % (2 * PAIR)) * K::kExp, lane);
    gv = gnext;
    __syncthreads();
    if (dot) {
      if (tid < n) {
        float d = 0.0f;
        for (int w = 0; w < NW; ++w) d += dots[w * C + tid];
        J.dot[((long long)slab * a.H + hd) * a.rows + s.row0 + at + tid] = d;
      }
      wb += (int64_t)dir * wst;
    }
    ob += (int64_t)dir * ost;
    at += dir;
    n = REV ? C : s.len - at;
  }

  if (!(REV ? s.first : s.last)) return;
  if ((MODE == kLaFwd || MODE == kLaV) && J.s_fin) la_store_state<K::KT>(S, J.s_fin + unit * a.state, J.sm, J.sn, J.DK, J.DV, col, h);
  if (MODE == kLaQ && J.xd_out) {
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

// JOBS: the modes of its jobs, a bit each.  With those of q and k the compiler
// keeps 83 to 135 scalar registers, mostly the jobs' arguments, in lanes of vector ones (forwards 0 to 8).
template <typename T, int DKP, int NW, int JOBS>
__global__ __launch_bounds__(NW * 64)
    __attribute__((amdgpu_waves_per_eu(LaTile<T, DKP, NW>::kWaves))) void
    pdssm_linattn_kernel(const LaArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const unsigned id = la_block(a.row);
  if (id == 0 && threadIdx.x < 2) a.header[threadIdx.x] = 0;
  LaUnit u;
  la_unit(a, id, u);
  if (u.sid >= a.segs) return;
  const LaJob& J = a.job[u.job];
  LaSeg s;
  if (!la_segment(a, u.sid, s)) return;
  if constexpr (JOBS & 1 << kLaFwd) la_body<T, DKP, NW, kLaFwd>(a, J, s, u.sid, u.hd, u.slab, smem);
  if constexpr (JOBS & 1 << kLaQ)
    if (J.mode == kLaQ) la_body<T, DKP, NW, kLaQ>(a, J, s, u.sid, u.hd, u.slab, smem);
  if constexpr (JOBS & 1 << kLaK)
    if (J.mode == kLaK) la_body<T, DKP, NW, kLaK>(a, J, s, u.sid, u.hd, u.slab, smem);
  if constexpr (JOBS & 1 << kLaV)
    if (J.mode == kLaV) la_body<T, DKP, NW, kLaV>(a, J, s, u.sid, u.hd, u.slab, smem);
}

// Contribution of one segment to the state behind it (before it, for a
// reversed job), written at that segment's place.  Reading y and z is its time
// (16 x 2048 steps, 24 heads, 64/32 bf16: 35 us, 212 MB behind the L2s at 6.0 TB/s; 65536 steps,
// 16 heads, 128/128: 120 us, 587 MB at 4.9; two chunks under way instead of one: the same).  The last segment in the
// job's direction has none behind it and does nothing.
//
// It goes through its chunks from that end on, each weighted with the decay f
// of all that lie between: the state needs no rescaling, chunks behind a decay
// that leaves nothing (f = 0) are not read, and what it reads last is what the
// product kernel starts with, still in the caches.
template <typename T, int DKP, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(LaTile<T, DKP, NW>::kStateWaves))) void
pdssm_linattn_state_kernel(const LaArgs a) {
  using K = LaTile<T, DKP, NW>;
  using F = typename T::frag;
  constexpr int C = K::C;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5,
            n32 = lane & 31;
  float* ew = (float*)(smem + 2 * (K::kX + K::kZ)) + wave * 64;   // this wave's own copy of the weights
  LaUnit u;
  la_unit(a, la_block(a.row), u);
  if (u.sid >= a.segs) return;
  const int slab = u.slab, hd = u.hd, sid = u.sid;
  const LaJob& J = a.job[u.job];
  LaSeg s;
  if (!la_segment(a, sid, s)) return;
  const int rev = J.rev;
  if (rev ? s.first : s.last) return;
  const int slab0 = slab * NW * 32, col = slab0 + wave * 32 + la_pi(n32);
  const int chunks = (s.len + C - 1) / C;
  const int first = rev ? 0 : (chunks ? chunks - 1 : 0) * C;
  typename K::X ty;
  typename K::Z tz;
  ty.init(la_ptr<T>(J.y, s.vb, hd / J.yd, s.t0 + first), J.y.st, tid, J.DK);
  tz.init(la_ptr<T>(J.z, s.vb, hd / J.zd, s.t0 + first) + slab0, J.z.st, tid, J.DV - slab0);
  const int64_t dir = rev ? C : -C;
  const int64_t dy = dir * J.y.st * K::ES, dz = dir * J.z.st * K::ES, dg = dir * a.g.st;
  const bool whole = J.DK == DKP && J.DV - slab0 >= NW * 32;
  const float* gp = (const float*)a.g.p + (int64_t)s.vb * a.g.sb + (int64_t)hd * a.g.sh +
                    (int64_t)(s.t0 + first) * a.g.st;
  const int64_t goff = (lane & (C - 1)) * a.g.st + (lane / C) * dg;
  const float s_upd = J.s_upd;
  float gv = 0.0f;
  constexpr int PAIR = K::PAIR;
  auto fetch = [&](int n) {
    ty.fetch(n);
    tz.fetch(n);
  };
  auto fetch_g = [&](int n, int rest) { gv = (lane & (C - 1)) < (lane < C ? n : rest) ? gp[goff] : 0.0f; };
  double sum = 0.0;      // log2 of f
  // Weights of the next 64 / C chunks.  Every wave forms them for itself: one
  // wave would do it in the others' way, and they find room between the
  // matrix instructions.
  auto weights = [&]() {
    const double G = la_scan<C>(gv);
    double tot = la_lane(G, 63), before = sum;
    sum += tot;
    if (C == 32) {
      const double t0 = la_lane(G, 31);
      sum += t0;
      if (lane < 32)
        tot = t0;
      else
        before += t0;
    }
    ew[lane] = la_exp2((rev ? G : tot - G) + before) * s_upd;
  };
  if (chunks) {
    fetch_g(s.len - first, rev ? s.len - C : first);
    fetch(s.len - first);
  }
  la_f16 S[K::KT];
#pragma unroll
  for (int t = 0; t < K::KT; ++t) S[t] = la_f16{};
  uint32_t ycol = T::template col_base<K::XB>(lane, 0);
  uint32_t zcol = T::template col_base<K::ZB>(lane, wave * 32);
  weights();
  int n = s.len - first, at = first;
  bool more = chunks > 0;
  for (int q = 0; more; ++q) {
    if (n > C) n = C;
    asm volatile("" : "+v"(ycol), "+v"(zcol));
    // two places for the tiles: one barrier a chunk
    unsigned char* Y = smem + (q & 1) * (K::kX + K::kZ);
    unsigned char* Z = Y + K::kX;
    ty.commit(Y, tid, n, whole && n == C);
    tz.commit(Z, tid, n, whole && n == C);
    __syncthreads();
    if (q + 1 < chunks) {
      ty.base += dy;
      tz.base += dz;
      gp += dg;
      if (q % PAIR == PAIR - 1) fetch_g(rev ? s.len - at - C : C, rev ? s.len - at - 2 * C : at - C);   // waited for first
      fetch(rev ? s.len - at - C : C);
    } else {
      gv = 0.0f;
    }
    F zf[C / 16];
#pragma unroll
    for (int js = 0; js < C / 16; ++js) zf[js] = T::template col<K::ZB, K::ZP>(Z, zcol, 16 * js, 0);
    la_update<T, DKP, NW, true, K::kApart>(S, Y, ycol, zf, ew + q % PAIR * C, 1.0f, lane);
    at += (int)dir;
    n = rev ? s.len - at : C;
    more = q + 1 < chunks;
    if (q % PAIR == PAIR - 1) {
      more = more && !(__builtin_amdgcn_readfirstlane((int)(sum < -200.0)));   // f = 0
      weights();
    }
  }
  const long long to = ((long long)(sid + (rev ? -1 : 1)) * a.H + hd);
  la_store_state<K::KT>(S, J.seg_out + to * a.state, J.sm, J.sn, J.DK, J.DV, col, h);
  if (slab == 0 && tid == 0) J.seg_decay[to] = la_exp2(sum);
}

}  // namespace pdscan
