// Launchers of the linear-attention passes, and their small kernels: the
// segment table of packed sequences, the carry between segments, the
// log-decay gradient, the sum over heads that share a query or key head, and
// the single-token step.
#include <cfloat>

#include "pdscan_linattn.h"
#include "pdscan_linattn_launch.h"
#include "pdscan_linattn_table.h"

namespace pdscan {

// Entering states of all segments of a sequence and head from the segments'
// contributions, in place, four state elements a thread and eight segments'
// loads at once.  It moves every segment's state twice, at the rate of the
// cache behind the L2s (65536 steps in 32 segments, 16 heads, 128/128: 67 MB in
// 11.7 us).
__global__ __launch_bounds__(256) void pdssm_linattn_carry_kernel(LaCarryArgs a) {
  const LaCarry& c = a.c[blockIdx.z / a.tiles];
  const unsigned unit = la_block(a.row);
  const int b = unit / a.H, h = unit % a.H;
  const long long e = ((long long)(blockIdx.z % a.tiles) * 256 + threadIdx.x) * 4;
  if (b >= a.B || e >= a.state) return;
  const int s0 = a.starts ? a.starts[b] : b * a.nseg;
  const int s1 = a.starts ? a.starts[b + 1] : s0 + a.nseg;
  const int n = s1 - s0 - 1;
  float4 S = make_float4(0, 0, 0, 0);
  if (c.user) S = *(const float4*)(c.user + ((long long)b * a.H + h) * a.state + e);
  constexpr int U = 8;
  for (int i0 = 0; i0 < n; i0 += U) {
    float4 v[U];
    float d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u < n ? i0 + u : n - 1;
      const long long at = (long long)(c.rev ? s1 - 2 - i : s0 + 1 + i) * a.H + h;
      v[u] = *(const float4*)(c.seg + at * a.state + e);
      d[u] = c.decay[at];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= n) break;
      const long long at = (long long)(c.rev ? s1 - 2 - (i0 + u) : s0 + 1 + i0 + u) * a.H + h;
      S.x = d[u] * S.x + v[u].x;
      S.y = d[u] * S.y + v[u].y;
      S.z = d[u] * S.z + v[u].z;
      S.w = d[u] * S.w + v[u].w;
      *(float4*)(c.seg + at * a.state + e) = S;
    }
  }
}

__device__ __forceinline__ double block_sum(double x, double* red, int tid) {
#pragma unroll
  for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m, 64);
  __syncthreads();
  if ((tid & 63) == 0) red[tid >> 6] = x;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// This thread's part of the product of two states.
__device__ __forceinline__ double la_dot_states(const float* a, const float* b, long long n, int tid) {
  double x = 0.0;
#pragma unroll 4
  for (int e = tid; e < (int)(n / 4); e += kLaPiece) {
    const float4 p = ((const float4*)a)[e], q = ((const float4*)b)[e];
    x += (double)((p.x * q.x + p.y * q.y) + (p.z * q.z + p.w * q.w));
  }
  return x;
}

// d loss / d log a_t of one segment and head.  Pairs (key at or before t-1,
// query at or behind t) meet at t, so with r_i = q_i . dq_i (every key before
// query i, its own left out) and c_j = k_j . dk_j (every query behind key j)
//   g_t = sum_{i >= t} r_i - sum_{j >= t} c_j + <S_end, dS_end>
// over the rest of the segment: pairs inside it cancel but for those that
// meet at t, and the last term holds those that meet behind its end.  The
// sums run in 64 bits, but r and c carry fp32 errors that do not cancel and
// grow with the square root of their number: hence the at most 512 steps of a segment.
//
// Over the whole segment the sum is <S_start, dS_start>, the product of the states
// before it.  What it differs by is the errors' sum; it is taken out along the
// segment in proportion to the squares of the terms, which leaves the
// errors of a walk held at both ends (a third of their squares on average, a
// quarter in the sum over t that a decay per head has).  Without h0's gradient
// the start of a sequence with an h0 is not known, and its first segment is held at its end alone.
// Errors of the norm so, and held at the end alone: 4 x 1024 steps, 4 heads, 64/32 bf16 2.4e-7
// and 4.1e-7, 8190 packed rows of 128/128 5.6e-7 and 8.0e-7.
//
// One step a thread: a segment is one round of the workgroup.  It reads three
// floats a step and four states a segment (24 heads, 16 x 2048 steps, 64/32: 22 us).
__global__ __launch_bounds__(kLaPiece) void pdssm_linattn_decay_kernel(const LaDecayArgs a) {
  constexpr int W = kLaPiece / 64;
  __shared__ double red[4][W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const unsigned id = la_block(a.c.row);
  const int h = id % a.c.H, sid = id / a.c.H;
  if (sid >= a.c.segs) return;
  LaSeg s;
  if (!la_segment(a.c, sid, s)) {
    if (a.per_head && tid == 0) a.part[(long long)sid * a.c.H + h] = 0.0;
    return;
  }
  const int t = s.len - 1 - tid;
  const long long n = a.c.state, unit = (long long)s.b * a.c.H + h, seg = (long long)sid * a.c.H + h;
  double d = 0.0, v = 0.0, x = 0.0, y = 0.0;   // r - c, their squares, the products at the end and at the start
  // Where the decay is zero in fp32 (e^-104 < 2^-150), or no state lies before
  // the token, the product is zero: not left to what the sums' errors leave.
  bool none = t < 0 || (t == 0 && s.first && !a.h0);
  if (t >= 0) {
    none |= ((const float*)a.c.g.p)[(int64_t)s.vb * a.c.g.sb + (int64_t)h * a.c.g.sh + (int64_t)(s.t0 + t) * a.c.g.st] <
            -104.0f;
    const long long at = (long long)h * a.c.rows + s.row0 + t;
    const long long slab = (long long)a.c.H * a.c.rows;
    double r = 0.0, c = 0.0;
    for (int w = 0; w < a.slabs; ++w) {
      r += (double)a.r[w * slab + at];
      c += (double)a.k[w * slab + at];
    }
    d = r - c;
    v = r * r + c * c;
  }
  if (!s.last)
    x = la_dot_states(a.sS + (seg + a.c.H) * n, a.sR + seg * n, n, tid);
  else if (a.xd && tid < a.slabs)
    x = a.xd[((long long)tid * a.c.segs + sid) * a.c.H + h];
  const bool held = !s.first || !a.h0 || a.g_h0;
  if (!s.first)
    y = la_dot_states(a.sS + seg * n, a.sR + (seg - a.c.H) * n, n, tid);
  else if (a.h0 && a.g_h0)
    y = la_dot_states(a.h0 + unit * n, a.g_h0 + unit * n, n, tid);
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double up = __shfl_up(d, m, 64), uv = __shfl_up(v, m, 64);
    if (lane >= m) {
      d += up;
      v += uv;
    }
  }
#pragma unroll
  for (int m = 32; m; m >>= 1) {
    x += __shfl_xor(x, m, 64);
    y += __shfl_xor(y, m, 64);
  }
  if (lane == 63) {
    red[0][wave] = d;
    red[1][wave] = v;
    red[2][wave] = x;
    red[3][wave] = y;
  }
  __syncthreads();
  double all = 0.0, squares = 0.0;
  x = y = 0.0;
  for (int w = 0; w < W; ++w) {
    if (w < wave) {
      d += red[0][w];
      v += red[1][w];
    }
    all += red[0][w];
    squares += red[1][w];
    x += red[2][w];
    y += red[3][w];
  }
  double g = d + x;
  const double off = all + x - y;
  squares += x * x + y * y;
  if (held && squares > 0.0) g -= off * ((v + x * x) / squares);
  if (none) g = 0.0;
  if (!a.per_head) {
    if (t >= 0)
      ((float*)a.out.p)[(int64_t)s.vb * a.out.sb + (int64_t)h * a.out.sh + (int64_t)(s.t0 + t) * a.out.st] = (float)g;
    return;
  }
#pragma unroll
  for (int m = 32; m; m >>= 1) g += __shfl_xor(g, m, 64);
  __syncthreads();
  if (lane == 0) red[0][wave] = g;
  __syncthreads();
  if (tid == 0) {
    double sum = 0.0;
    for (int w = 0; w < W; ++w) sum += red[0][w];
    a.part[seg] = sum;
  }
}

__global__ __launch_bounds__(256) void pdssm_linattn_decay_sum_kernel(const double* part, float* out, int H, int segs,
                                                                      unsigned row) {
  __shared__ double red[4];
  const unsigned h = la_block(row);
  if (h >= (unsigned)H) return;
  double x = 0.0;
  for (int s = threadIdx.x; s < segs; s += 256) x += part[(long long)s * H + h];
  x = block_sum(x, red, threadIdx.x);
  if (threadIdx.x == 0) out[h] = (float)x;
}

// Sum over the value heads of a query or key head, of g_q (y = 0) and g_k:
// each partial gradient read once (8190 rows, 16 heads on 4, 128: 151 MB in 25 us).
template <typename T>
__global__ __launch_bounds__(256) void pdssm_linattn_fold_kernel(const LaFoldArgs a) {
  const float* part = blockIdx.y ? a.part_k : a.part_q;
  const LaView& out = blockIdx.y ? a.out_k : a.out_q;
  const int Hk = a.H / a.ratio, c4 = a.d / 4;
  long long r0 = 0, r1 = a.rows;
  if (a.cu) {   // rows outside the sequences stay as they are
    r0 = a.cu[0];
    r1 = a.cu[a.B];
    r0 = r0 < 0 ? 0 : r0 > a.rows ? a.rows : r0;
    r1 = r1 < r0 ? r0 : r1 > a.rows ? a.rows : r1;
  }
  const long long n = (r1 - r0) * Hk * c4;
  for (long long q = (long long)blockIdx.x * 256 + threadIdx.x; q < n; q += (long long)gridDim.x * 256) {
    const int c = (int)(q % c4) * 4;
    const int hk = (int)(q / c4 % Hk);
    const long long row = r0 + q / c4 / Hk;
    const float* p = part + (row * a.H + (long long)hk * a.ratio) * a.d + c;
    float v[4] = {0, 0, 0, 0};
    for (int r = 0; r < a.ratio; ++r) {
      const float4 w = *(const float4*)(p + (long long)r * a.d);
      v[0] += w.x; v[1] += w.y; v[2] += w.z; v[3] += w.w;
    }
    const int64_t b = a.cu ? 0 : row / a.L, t = a.cu ? row : row % a.L;
    T::store4((typename T::store*)out.p + b * out.sb + hk * out.sh + t * out.st + c, v);
  }
}

// One token: S = a S + k v^T in place, o = s S^T q.  One workgroup owns `cols`
// value columns of one row and head; a thread owns four columns of every
// nr-th state row.  The state is read and written once, which is all the time
// (250 rows, 16 heads, 128/128: 532 MB in 95 us, 5.6 TB/s; one row: 5.0 us, of
// which the loads' way there and back is most).
template <typename T>
__global__ __launch_bounds__(256) void pdssm_linattn_step_kernel(const LaStepArgs a) {
  __shared__ float qs[kLaMaxD], ks[kLaMaxD];
  __shared__ __align__(16) float red[256 * 4];
  __shared__ int dup;
  const int tid = threadIdx.x;
  const int tiles = (a.dv + a.cols - 1) / a.cols;
  unsigned id = la_block(a.row);
  const int tile = id % tiles;
  id /= tiles;
  const int h = id % a.H, b = id / a.H;
  if (b >= a.B) return;
  const int c0 = tile * a.cols;
  const int cols = a.dv - c0 < a.cols ? a.dv - c0 : a.cols;
  using E = typename T::store;
  const int slot = a.idx ? a.idx[b] : b;
  E* op = (E*)a.o.p + (int64_t)b * a.o.sb + (int64_t)h * a.o.sh + c0;
  if (slot < 0 || slot >= a.slots) {
    // an empty row gives zeros; a slot past the pool gives NaN
    const float f = slot < 0 ? 0.0f : __builtin_nanf("");
    const float v[4] = {f, f, f, f};
    for (int c = tid * 4; c < cols; c += 1024) T::store4(op + c, v);
    return;
  }
  if (tid == 0) dup = 0;
  const E* qp = (const E*)a.q.p + (int64_t)b * a.q.sb + (int64_t)(h / a.qd) * a.q.sh;
  const E* kp = (const E*)a.k.p + (int64_t)b * a.k.sb + (int64_t)(h / a.qd) * a.k.sh;
  for (int c = tid * 4; c < a.dk; c += 1024) {
    T::load4(qp + c, qs + c);
    T::load4(kp + c, ks + c);
  }
  __syncthreads();
  if (a.idx) {
    // a slot named twice: the first row has it
    int found = 0;
    for (int r = tid; r < b; r += 256) found |= a.idx[r] == slot;
    if (found) dup = 1;
    __syncthreads();
    if (dup) {
      const float f = __builtin_nanf("");
      const float v[4] = {f, f, f, f};
      for (int c = tid * 4; c < cols; c += 1024) T::store4(op + c, v);
      return;
    }
  }
  const int W = cols / 4, nr = 256 / W;
  const int rg = tid / W, c = tid % W * 4;
  const float decay = expf(((const float*)a.g.p)[(int64_t)b * a.g.sb + (int64_t)h * a.g.sh]);
  float o[4] = {0, 0, 0, 0};
  if (rg < nr) {
    float v[4];
    T::load4((const E*)a.v.p + (int64_t)b * a.v.sb + (int64_t)h * a.v.sh + c0 + c, v);
    float* st = a.state + ((int64_t)slot * a.H + h) * a.dk * a.dv + c0 + c;
#pragma unroll 8
    for (int r = rg; r < a.dk; r += nr) {
      float4 x = *(float4*)(st + (int64_t)r * a.dv);
      const float kk = ks[r], qq = qs[r];
      x.x = decay * x.x + kk * v[0];
      x.y = decay * x.y + kk * v[1];
      x.z = decay * x.z + kk * v[2];
      x.w = decay * x.w + kk * v[3];
      *(float4*)(st + (int64_t)r * a.dv) = x;
      o[0] += qq * x.x; o[1] += qq * x.y; o[2] += qq * x.z; o[3] += qq * x.w;
    }
    *(float4*)(red + 4 * tid) = make_float4(o[0], o[1], o[2], o[3]);
  }
  __syncthreads();
  // The nr partial sums of a column: more than 16 in two rounds, by eight
  // threads in the first (64 of them 5.7 -> 5.0 us for the call; 16 4.1 -> 4.4).
  int parts = nr;
  if (nr > 16) {
    parts = 8;
    if (rg < parts) {
      for (int g = rg + parts; g < nr; g += parts) {
        const float4 p = *(const float4*)(red + 4 * (g * W + c / 4));
        o[0] += p.x; o[1] += p.y; o[2] += p.z; o[3] += p.w;
      }
      *(float4*)(red + 4 * tid) = make_float4(o[0], o[1], o[2], o[3]);
    }
    __syncthreads();
  }
  if (tid < W) {
    float x[4] = {0, 0, 0, 0};
    for (int g = 0; g < parts; ++g) {
      const float4 p = *(const float4*)(red + 4 * (g * W + tid));
      x[0] += p.x; x[1] += p.y; x[2] += p.z; x[3] += p.w;
    }
    for (int e = 0; e < 4; ++e) x[e] *= a.scale;
    T::store4(op + c, x);
  }
}

hipError_t launch_linattn_step(const LaStepArgs& args, hipStream_t st) {
  LaStepArgs a = args;
  const int tiles = (a.dv + a.cols - 1) / a.cols;
  const LaGrid g = la_grid_rows((long long)a.B * a.H * tiles, 256);
  a.row = g.x;
  if (a.bf16)
    hipLaunchKernelGGL(pdssm_linattn_step_kernel<LaBf16>, dim3(g.x, g.y), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(pdssm_linattn_step_kernel<LaF32>, dim3(g.x, g.y), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_linattn_table(const int32_t* cu, int32_t* table, int32_t* starts, int B, int L, int seg, int segs,
                                hipStream_t st) {
  hipLaunchKernelGGL(pdssm_linattn_table_kernel, dim3(1), dim3(256), 0, st, cu, table, starts, B, L, seg, segs);
  return hipGetLastError();
}

hipError_t launch_linattn_carry(const LaCarryArgs& args, int passes, hipStream_t st) {
  LaCarryArgs a = args;
  const LaGrid g = la_grid_rows((long long)a.B * a.H, 256);
  a.row = g.x;
  hipLaunchKernelGGL(pdssm_linattn_carry_kernel, dim3(g.x, g.y, a.tiles * passes), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_linattn_decay(const LaDecayArgs& args, hipStream_t st) {
  LaDecayArgs a = args;
  LaGrid g = la_grid_rows((long long)a.c.segs * a.c.H, kLaPiece);
  a.c.row = g.x;
  hipLaunchKernelGGL(pdssm_linattn_decay_kernel, dim3(g.x, g.y), dim3(kLaPiece), 0, st, a);
  if (a.per_head) {
    g = la_grid_rows(a.c.H, 256);
    hipLaunchKernelGGL(pdssm_linattn_decay_sum_kernel, dim3(g.x, g.y), dim3(256), 0, st, a.part, (float*)a.out.p, a.c.H,
                       a.c.segs, g.x);
  }
  return hipGetLastError();
}

hipError_t launch_linattn_fold(const LaFoldArgs& a, hipStream_t st) {
  const long long n = a.rows * (a.H / a.ratio) * (a.d / 4);
  long long grid = (n + 255) / 256;
  if (grid > 8192) grid = 8192;
  if (grid < 1) grid = 1;
  if (a.bf16)
    hipLaunchKernelGGL(pdssm_linattn_fold_kernel<LaBf16>, dim3((unsigned)grid, 2), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(pdssm_linattn_fold_kernel<LaF32>, dim3((unsigned)grid, 2), dim3(256), 0, st, a);
  return hipGetLastError();
}

// The product kernels, by type, x-row width and waves.
hipError_t launch_linattn_form(const LaArgs& args, int bf16, int pass, hipStream_t st) {
  LaArgs a = args;
  const int dk = la_pad(a.job[0].DK), nw = la_waves(a.job[0].DK, a.job[0].DV, bf16);
  const LaGrid g = la_grid_rows(la_grid(a), 64 * nw);
  a.row = g.x;
  if (bf16)
    return dk == 32    ? la_bf16_32(a, nw, pass, g, st)
           : dk == 64  ? la_bf16_64(a, nw, pass, g, st)
           : dk == 128 ? la_bf16_128(a, nw, pass, g, st)
                       : la_bf16_256(a, nw, pass, g, st);
  return dk == 32    ? la_f32_32(a, nw, pass, g, st)
         : dk == 64  ? la_f32_64(a, nw, pass, g, st)
         : dk == 128 ? la_f32_128(a, nw, pass, g, st)
                     : la_f32_256(a, nw, pass, g, st);
}

}  // namespace pdscan
