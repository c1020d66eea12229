// Element types, rounding and the few functions that the kernels of the
// selective scan, the convolution and the norm share.
#pragma once

#include <hip/hip_runtime.h>

#include "pdscan_ssm_plan.h"

namespace pdscan {

typedef __bf16 ss_bf2 __attribute__((ext_vector_type(2)));
typedef float ss_f2 __attribute__((ext_vector_type(2)));

// V neighbouring elements, loaded and stored at once.
template <typename E, int V>
struct alignas(sizeof(E) * V > 16 ? 16 : sizeof(E) * V) SsVec {
  E e[V];
};

struct SsF32 {
  using E = float;
  static __device__ __forceinline__ float get(float x) { return x; }
  template <int V>
  static __device__ __forceinline__ void put(SsVec<E, V>& o, const float* x) {
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = x[i];
  }
};
struct SsBf16 {
  using E = uint16_t;
  static __device__ __forceinline__ float get(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
  // rounded to the nearest, once, from the fp32 value
  template <int V>
  static __device__ __forceinline__ void put(SsVec<E, V>& o, const float* x) {
    if constexpr (V == 1) {
      o.e[0] = __builtin_bit_cast(uint16_t, (__bf16)x[0]);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const uint32_t u = __builtin_bit_cast(uint32_t, __builtin_convertvector(ss_f2{x[i], x[i + 1]}, ss_bf2));
        o.e[i] = (uint16_t)u;
        o.e[i + 1] = (uint16_t)(u >> 16);
      }
    }
  }
};

template <typename T, int V>
__device__ __forceinline__ SsVec<typename T::E, V> ss_load(const void* p, int64_t at) {
  return *(const SsVec<typename T::E, V>*)((const typename T::E*)p + at);
}
template <typename T, int V>
__device__ __forceinline__ void ss_store(void* p, int64_t at, const float* x) {
  SsVec<typename T::E, V> o;
  T::template put<V>(o, x);
  *(SsVec<typename T::E, V>*)((typename T::E*)p + at) = o;
}

// V neighbouring elements on their way, as the words that they come in: what
// unpacks them stays behind the wait for them.
template <typename T, int V>
struct SsRaw {
  static constexpr int kBytes = V * (int)sizeof(typename T::E), kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(typename T::E) == 4) return __builtin_bit_cast(float, w[i]);
    return __builtin_bit_cast(float, i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};
// Addressed by one uniform pointer, which walks with the tiles, and this
// lane's 32 bits of offset (kept from being added up ahead of the loop: half the
// registers of a pointer a lane).
template <typename T, int V>
__device__ __forceinline__ void ss_load_at(SsRaw<T, V>& r, const char* tile, uint32_t off) {
  asm("" : "+v"(off));
  if constexpr (SsRaw<T, V>::kBytes == 2) {
    r.w[0] = *(const uint16_t*)(tile + off);
  } else {
    using Q = SsVec<uint32_t, SsRaw<T, V>::kWords>;
    const Q q = *(const Q*)(tile + off);
#pragma unroll
    for (int i = 0; i < SsRaw<T, V>::kWords; ++i) r.w[i] = q.e[i];
  }
}
// The thread's number as a value of its own: what follows from it is formed
// where it stands, not ahead of a loop.
__device__ __forceinline__ int ss_thread_here() {
  int i = threadIdx.x;
  asm volatile("" : "+v"(i));
  return i;
}
// Waits here for what is on its way.
template <typename T, int V>
__device__ __forceinline__ void ss_arrived(SsRaw<T, V>& r) {
#pragma unroll
  for (int i = 0; i < SsRaw<T, V>::kWords; ++i) asm volatile("" : "+v"(r.w[i]));
}
template <typename T, int V>
__device__ __forceinline__ void ss_load_raw(SsRaw<T, V>& r, const void* p, int64_t at) {
  using Q = SsVec<uint32_t, SsRaw<T, V>::kWords>;
  const Q q = *(const Q*)((const typename T::E*)p + at);
#pragma unroll
  for (int i = 0; i < SsRaw<T, V>::kWords; ++i) r.w[i] = q.e[i];
}
template <typename T, int V>
__device__ __forceinline__ void ss_store_raw(void* p, int64_t at, const SsRaw<T, V>& r) {
  using Q = SsVec<uint32_t, SsRaw<T, V>::kWords>;
  Q q;
#pragma unroll
  for (int i = 0; i < SsRaw<T, V>::kWords; ++i) q.e[i] = r.w[i];
  *(Q*)((typename T::E*)p + at) = q;
}
template <typename T, int V>
__device__ __forceinline__ void ss_store_at(char* tile, uint32_t off, const float* x) {
  asm("" : "+v"(off));
  SsVec<typename T::E, V> o;
  T::template put<V>(o, x);
  *(SsVec<typename T::E, V>*)(tile + off) = o;
}
template <typename T>
__device__ __forceinline__ char* ss_tile_at(const LaView& v, int64_t vb, int64_t row, int64_t c) {
  return (char*)v.p + (vb * v.sb + row * v.st + c) * (int64_t)sizeof(typename T::E);
}
template <typename T>
__device__ __forceinline__ uint32_t ss_off(const LaView& v, int row, int c) {
  return ((uint32_t)row * (uint32_t)v.st + (uint32_t)c) * (uint32_t)sizeof(typename T::E);
}
// The same, formed where it stands: a register less to hold through a loop.
// (Rows of a tile and step strides, at most 2^23, are within 24 bits.)
template <typename T>
__device__ __forceinline__ uint32_t ss_off_here(const LaView& v, int row, int c) {
  asm volatile("" : "+v"(row));
  return (__umul24((uint32_t)row, (uint32_t)v.st) + (uint32_t)c) * (uint32_t)sizeof(typename T::E);
}
// Bytes of `rows` rows.
template <typename T>
__device__ __forceinline__ int64_t ss_rows(const LaView& v, int rows) {
  return v.st * rows * (int64_t)sizeof(typename T::E);
}

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kLn2Rest = (float)(0.69314718055994530942 - (double)kLn2);   // what fp32 drops of ln 2

__device__ __forceinline__ float ss_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// What goes into a decay's exponent, a sum of steps or A log2 e, ends at fp32's
// largest number: were it infinite, its product with a decay or a step of zero would
// not be a number.  One instruction each (steps are not negative, A is not positive).
constexpr float kMost = 3.40282347e38f;
__device__ __forceinline__ float ss_held_sum(float x) { return __builtin_elementwise_minimum(x, kMost); }
__device__ __forceinline__ float ss_held_decay(float x) { return __builtin_elementwise_maximum(x, -kMost); }

// e^-|x|, to a step of fp32 or two: 2^t with t = n log2 e rounded, times e^r, 1 + r, of
// what is left, r = n - t ln 2 with ln 2 in two parts (Cody and Waite's reduction; with
// one part r would be .05 |x| half steps off, left out altogether |x| of them).  It is zero from |x|
// = 104 on, and |x| ends at 128: past 2.4e38 t would be infinite, r too, and zero times
// that not a number (a type's lowest value switches a token off).  One
// instruction, which passes on what is not a number as fmaxf would not.
__device__ __forceinline__ float ss_decay(float x) {
  const float n = __builtin_elementwise_maximum(-fabsf(x), -128.0f), t = kLog2e * n, e = ss_exp2(t);
  return __builtin_fmaf(e, __builtin_fmaf(-t, kLn2Rest, __builtin_fmaf(-t, kLn2, n)), e);
}
// 1 / (1 + e^-x) from e = e^-|x|.
__device__ __forceinline__ float ss_sigmoid_of(float x, float e) {
  return (x >= 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e);
}
// The gate's: bf16 takes the short way, off by |x| steps of fp32 at most (x = -20: 2^-20).
template <typename T>
__device__ __forceinline__ float ss_sigmoid(float x) {
  if constexpr (sizeof(typename T::E) == 2) return __builtin_amdgcn_rcpf(1.0f + ss_exp2(-kLog2e * x));
  return ss_sigmoid_of(x, ss_decay(x));
}

// log(1 + e^x) = max(x, 0) + log1p(e) with e = e^-|x|.  log1p(e) is log(w),
// w = 1 + e rounded, and what the rounding dropped, e - (w - 1): small steps keep
// their digits (dividing that by w would change less than 2^-24 of e).
__device__ __forceinline__ float ss_softplus_of(float x, float e) {
  const float w = 1.0f + e;
  return fmaxf(x, 0.0f) + __builtin_fmaf(kLn2, __builtin_amdgcn_logf(w), e - (w - 1.0f));
}

// Steps of V cells, their slopes (sg[v]) where asked for, and zero behind the
// end.  The cells side by side in one uniform branch: taken one by one, each
// would wait for its own exponential and logarithm.
template <int V, bool SLOPE>
__device__ __forceinline__ void ss_steps(float (&d)[V], float (&sg)[V], int softplus, bool live) {
  if (softplus) {
    float e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = ss_decay(d[v]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (SLOPE) sg[v] = ss_sigmoid_of(d[v], e[v]);
      d[v] = ss_softplus_of(d[v], e[v]);
    }
  } else if (SLOPE) {
#pragma unroll
    for (int v = 0; v < V; ++v) sg[v] = 1.0f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    asm("" : "+v"(d[v]));   // (kept out of a branch on `live`)
    d[v] = live ? d[v] : 0.0f;
  }
}

template <int CTRL>
__device__ __forceinline__ float ss_dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppRor4 = 0x124, kDppRor8 = 0x128,
              kDppShl4 = 0x104;

// Exchanges across a wave, by hand, as the compiler's builtins give the first
// result twice; each waits for the two states that it has to be behind what wrote
// its operands, four exchanges at a time where there are as many.
//   32: a's upper half and b's lower one change places;
//   16: a's odd rows of 16 lanes and b's even ones.
// So a + b is then the sum over lanes 32 apart of a in the lower half, of b in
// the upper; over rows next to each other of a in even rows, of b in odd ones.
__device__ __forceinline__ float ss_fold32(float a, float b) {
  asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(a), "+v"(b));
  return a + b;
}
__device__ __forceinline__ float ss_fold16(float a, float b) {
  asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(a), "+v"(b));
  return a + b;
}
// r[i] = fold(a[i], b[i]), N even.
template <int N>
__device__ __forceinline__ void ss_fold32(float (&r)[N], float (&a)[N], float (&b)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += N < 4 ? 2 : 4) {
    if constexpr (N < 4)
      asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\tv_permlane32_swap_b32 %2, %3" : "+v"(a[i]), "+v"(b[i]), "+v"(a[i + 1]), "+v"(b[i + 1]));
    else
      asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\tv_permlane32_swap_b32 %2, %3\n\t"
          "v_permlane32_swap_b32 %4, %5\n\tv_permlane32_swap_b32 %6, %7"
          : "+v"(a[i]), "+v"(b[i]), "+v"(a[i + 1]), "+v"(b[i + 1]), "+v"(a[i + 2]), "+v"(b[i + 2]), "+v"(a[i + 3]), "+v"(b[i + 3]));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = a[i] + b[i];
}
template <int N>
__device__ __forceinline__ void ss_fold16(float (&r)[N], float (&a)[N], float (&b)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += N < 4 ? 2 : 4) {
    if constexpr (N < 4)
      asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1\n\tv_permlane16_swap_b32 %2, %3" : "+v"(a[i]), "+v"(b[i]), "+v"(a[i + 1]), "+v"(b[i + 1]));
    else
      asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1\n\tv_permlane16_swap_b32 %2, %3\n\t"
          "v_permlane16_swap_b32 %4, %5\n\tv_permlane16_swap_b32 %6, %7"
          : "+v"(a[i]), "+v"(b[i]), "+v"(a[i + 1]), "+v"(b[i + 1]), "+v"(a[i + 2]), "+v"(b[i + 2]), "+v"(a[i + 3]), "+v"(b[i + 3]));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = a[i] + b[i];
}
// Sums over the four rows of 16 lanes: row r of the result has v_r's.
__device__ __forceinline__ float ss_fold_rows(float v0, float v1, float v2, float v3) {
  float r[2], a[2] = {v0, v1}, b[2] = {v2, v3};
  ss_fold32(r, a, b);
  return ss_fold16(r[0], r[1]);
}

// Sum over P lanes next to each other, in every one of them (P: up to 64).
template <int P>
__device__ __forceinline__ float ss_sum(float x) {
  if constexpr (P >= 2) x += ss_dpp<kDppXor1>(x);
  if constexpr (P >= 4) x += ss_dpp<kDppXor2>(x);
  if constexpr (P >= 8) x += ss_dpp<kDppHalfMirror>(x);
  if constexpr (P >= 16) x += ss_dpp<kDppRor8>(x);
  if constexpr (P >= 32) x = ss_fold16(x, x);
  if constexpr (P >= 64) x = ss_fold32(x, x);
  return x;
}

// The workgroup's number, in a launch of la_grid_rows.
__device__ __forceinline__ unsigned ss_block(unsigned row) { return blockIdx.y * row + blockIdx.x; }

// Whether row b of a step has no state of its own: a slot that is empty, past
// the pool, or an earlier row's.  Every wave searches for itself: 256 rows are
// four loads at once, and no wave waits for another.
__device__ __forceinline__ bool ss_taken(const int32_t* idx, int b, int slot, int slots, int lane) {
  if (slot < 0 || slot >= slots) return true;
  if (!idx) return false;
  int found = 0;
#pragma unroll 4
  for (int r = lane; r < b; r += 64) found |= idx[r] == slot;
  return __any(found);
}

struct SsSeg {
  int b, t0, len;                // sequence; first row of the step axis, rows
  int64_t vb;                    // row of the batch axis
  bool first, last;
};

__device__ __forceinline__ bool ss_segment(const SsSegs& g, int sid, SsSeg& s) {
  auto one = [](int x) { return __builtin_amdgcn_readfirstlane(x); };   // (the same in every lane)
  if (g.table) {
    const int4 e = *(const int4*)(g.table + 4 * (int64_t)sid);
    if (one(e.z) < 0) return false;
    s.b = one(e.x);
    s.t0 = one(e.y);
    s.len = one(e.z);
    s.first = one(e.w) & 1;
    s.last = one(e.w) >> 1;
    s.vb = 0;
  } else if (g.cu) {
    s.b = sid;
    int t0 = one(g.cu[sid]), t1 = one(g.cu[sid + 1]);
    t0 = t0 < 0 ? 0 : t0 > g.L ? g.L : t0;
    t1 = t1 < t0 ? t0 : t1 > g.L ? g.L : t1;
    s.t0 = t0;
    s.len = t1 - t0;
    s.first = s.last = true;
    s.vb = 0;
  } else {
    s.b = sid / g.nseg;
    const int i = sid % g.nseg;
    s.t0 = i * g.seg;
    s.len = g.L - s.t0 < g.seg ? g.L - s.t0 : g.seg;
    s.first = i == 0;
    s.last = i == g.nseg - 1;
    s.vb = s.b;
  }
  return true;
}

}  // namespace pdscan
