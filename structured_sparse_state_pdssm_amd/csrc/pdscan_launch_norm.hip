// Norm over the rows of a block's heads, with its gate, residual and scale:
//
//   y = residual + s (w u / rms(u)) [silu(z)],  u = x, or x silu(z);  rms^2 = mean(u^2) + eps.
//
// Every cell is read and written once, which bounds it (24 heads of 32 at 32768
// tokens, gated, bf16: 151 MB in 31 us, 4.9 TB/s; gradient of 16384 rows of 512 in
// fp32: 172 MB in 32 us, 5.4 TB/s); a row is held in registers between its sum and its output.  P lanes share a row; lanes of a workgroup
// keep their columns over many rows, so weights are read once and their
// gradients are sums of a lane until its last row.  Backwards, with k = u / rms(u)
// and g the gradient of w k:
//   g_u = (w g - k mean(w g k)) / rms(u),  g_w = sum g k.
#include <type_traits>

#include "pdscan_ssm.h"
#include "pdscan_ssm_launch.h"

namespace pdscan {

enum { kNmNone, kNmBefore, kNmAfter };

template <int P>
__device__ __forceinline__ float nm_sum(float x, float* red, int tid) {
  if constexpr (P <= 64) return ss_sum<P>(x);
  x = ss_sum<64>(x);
  __syncthreads();
  if ((tid & 63) == 0) red[tid >> 6] = x;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

struct NmLane {
  int h, p, slot, chunk;
  bool ok;
};
template <int P>
__device__ __forceinline__ bool nm_lane(const NmArgs& a, NmLane& l) {
  const unsigned id = ss_block(a.row);
  const int col = id % a.tiles * a.cols + threadIdx.x % a.cols;
  l.chunk = id / a.tiles;
  l.slot = threadIdx.x / a.cols;
  l.h = col / P;
  l.p = col % P;
  l.ok = l.slot < a.slots && l.h < a.H;
  return l.chunk < a.chunks;
}

template <typename T, int P, int K>
__global__ __launch_bounds__(256) void pdssm_norm_kernel(const NmArgs a) {
  using E = typename T::E;
  constexpr int V = 16 / sizeof(E);
  __shared__ float red[4];
  NmLane l;
  if (!nm_lane<P>(a, l)) return;
  const int tid = threadIdx.x;
  float w[K][V], s[K][V];
  bool in[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * P + l.p) * V;
    in[k] = l.ok && c < a.d;
    const int64_t at = (a.per_head ? (int64_t)l.h * a.d : 0) + c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[k][v] = in[k] ? a.w[at + v] : 0.0f;
      s[k][v] = in[k] && a.s ? a.s[at + v] : 1.0f;
    }
  }
  const unsigned step = (unsigned)a.chunks * a.slots, rows = (unsigned)a.rows;   // (the host keeps both below 2^31)
  // (every lane of the workgroup makes the same rounds: sums of whole rows wait for each other)
  for (unsigned r0 = (unsigned)l.chunk * a.slots; r0 < rows; r0 += step) {
    const unsigned r = r0 + l.slot;
    const bool live = r < rows;
    const int64_t b = r / a.L, t = r % a.L;
    auto at = [&](const LaView& v, int k) { return b * v.sb + (int64_t)l.h * v.sh + t * v.st + (k * P + l.p) * V; };
    SsVec<E, V> xv[K] = {}, zv[K] = {}, rv[K] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!live || !in[k]) continue;
      xv[k] = ss_load<T, V>(a.x.p, at(a.x, k));
      if (a.gate != kNmNone) zv[k] = ss_load<T, V>(a.z.p, at(a.z, k));
      if (a.r.p) rv[k] = ss_load<T, V>(a.r.p, at(a.r, k));
    }
    float u[K][V], gate[K][V], q = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        u[k][v] = T::get(xv[k].e[v]);
        gate[k][v] = 1.0f;
        if (a.gate != kNmNone) {
          const float z = T::get(zv[k].e[v]);
          gate[k][v] = z * ss_sigmoid<T>(z);
          if (a.gate == kNmBefore) u[k][v] *= gate[k][v];
        }
        q = __builtin_fmaf(u[k][v], u[k][v], q);
      }
    q = nm_sum<P>(q, red, tid);
    const float rms = __builtin_amdgcn_rsqf(q / (float)a.d + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!live || !in[k]) continue;
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v] = u[k][v] * rms * w[k][v];
        if (a.gate == kNmAfter) o[v] *= gate[k][v];
        o[v] *= s[k][v];
        if (a.r.p) o[v] += T::get(rv[k].e[v]);
      }
      ss_store<T, V>(a.y.p, at(a.y, k), o);
    }
  }
}

template <typename T, int P, int K>
__global__ __launch_bounds__(256) void pdssm_norm_bwd_kernel(const NmArgs a) {
  using E = typename T::E;
  constexpr int V = 16 / sizeof(E);
  __shared__ float red[4];
  __shared__ float part[256 * V];
  if (ss_block(a.row) == 0 && threadIdx.x < 2) a.header[threadIdx.x] = 0;
  NmLane l;
  if (!nm_lane<P>(a, l)) return;
  const int tid = threadIdx.x;
  float w[K][V], s[K][V], gw[K][V] = {}, gs[K][V] = {};
  bool in[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * P + l.p) * V;
    in[k] = l.ok && c < a.d;
    const int64_t at = (a.per_head ? (int64_t)l.h * a.d : 0) + c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[k][v] = in[k] ? a.w[at + v] : 0.0f;
      s[k][v] = in[k] && a.s ? a.s[at + v] : 1.0f;
    }
  }
  const unsigned step = (unsigned)a.chunks * a.slots, rows = (unsigned)a.rows;   // (the host keeps both below 2^31)
  for (unsigned r0 = (unsigned)l.chunk * a.slots; r0 < rows; r0 += step) {
    const unsigned r = r0 + l.slot;
    const bool live = r < rows;
    const int64_t b = r / a.L, t = r % a.L;
    auto at = [&](const LaView& v, int k) { return b * v.sb + (int64_t)l.h * v.sh + t * v.st + (k * P + l.p) * V; };
    SsVec<E, V> xv[K] = {}, zv[K] = {}, gv[K] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!live || !in[k]) continue;
      xv[k] = ss_load<T, V>(a.x.p, at(a.x, k));
      gv[k] = ss_load<T, V>(a.gy.p, at(a.gy, k));
      if (a.gate != kNmNone) zv[k] = ss_load<T, V>(a.z.p, at(a.z, k));
    }
    // q = sum u^2, e = sum w g u
    float u[K][V], q = 0.0f, e = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        u[k][v] = T::get(xv[k].e[v]);
        float g = T::get(gv[k].e[v]) * s[k][v];
        if (a.gate != kNmNone) {
          const float z = T::get(zv[k].e[v]), gate = z * ss_sigmoid<T>(z);
          if (a.gate == kNmBefore) u[k][v] *= gate;
          else g *= gate;
        }
        q = __builtin_fmaf(u[k][v], u[k][v], q);
        e = __builtin_fmaf(w[k][v] * g, u[k][v], e);
      }
    q = nm_sum<P>(q, red, tid);
    e = nm_sum<P>(e, red, tid);
    const float rms = __builtin_amdgcn_rsqf(q / (float)a.d + a.eps), m = e * rms / (float)a.d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!live || !in[k]) continue;
      float ox[V], oz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float gy = T::get(gv[k].e[v]), kk = u[k][v] * rms;
        float g = gy * s[k][v], n = kk * w[k][v], gate = 1.0f, slope = 0.0f;
        if (a.gate != kNmNone) {
          const float z = T::get(zv[k].e[v]), sig = ss_sigmoid<T>(z);
          gate = z * sig;
          slope = sig * __builtin_fmaf(z, 1.0f - sig, 1.0f);
        }
        if (a.gate == kNmAfter) {
          oz[v] = g * n * slope;
          g *= gate;
          n *= gate;
        }
        gw[k][v] = __builtin_fmaf(g, kk, gw[k][v]);
        gs[k][v] = __builtin_fmaf(gy, n, gs[k][v]);
        ox[v] = rms * __builtin_fmaf(-kk, m, w[k][v] * g);
        if (a.gate == kNmBefore) {
          oz[v] = ox[v] * T::get(xv[k].e[v]) * slope;
          ox[v] *= gate;
        }
      }
      ss_store<T, V>(a.gx.p, at(a.gx, k), ox);
      if (a.gate != kNmNone) ss_store<T, V>(a.gz.p, at(a.gz, k), oz);
    }
  }
  // the rows' slots of this workgroup, in order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which && !a.s) break;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) part[tid * V + v] = which ? gs[k][v] : gw[k][v];
      __syncthreads();
      if (l.slot == 0 && in[k]) {
        float o[V] = {};
        for (int i = 0; i < a.slots; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] += part[(i * a.cols + tid) * V + v];
        float* to = a.part + l.chunk * a.part_chunk + l.h * a.part_head + which * a.part_s + (k * P + l.p) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) to[v] = o[v];
      }
    }
  }
}

namespace {

template <typename F>
void by_shape(int d, int bf16, F f) {
  const NmShape n = nm_shape(d, bf16);
#define PDSCAN_NM(p, k) f(std::integral_constant<int, p>{}, std::integral_constant<int, k>{})
  if (n.P == 256) {
    if (n.K == 2) PDSCAN_NM(256, 2);
    else if (n.K == 4) PDSCAN_NM(256, 4);
    else PDSCAN_NM(256, 8);
  } else if (n.P == 64) {
    if (n.K == 1) PDSCAN_NM(64, 1);
    else if (n.K == 2) PDSCAN_NM(64, 2);
    else PDSCAN_NM(64, 4);
  } else if (n.P == 32) PDSCAN_NM(32, 1);
  else if (n.P == 16) PDSCAN_NM(16, 1);
  else if (n.P == 8) PDSCAN_NM(8, 1);
  else if (n.P == 4) PDSCAN_NM(4, 1);
  else if (n.P == 2) PDSCAN_NM(2, 1);
  else PDSCAN_NM(1, 1);
#undef PDSCAN_NM
}

}  // namespace

hipError_t launch_norm_fwd(const NmArgs& args, int bf16, hipStream_t st) {
  NmArgs a = args;
  const LaGrid g = la_grid_rows((long long)a.tiles * a.chunks, 256);
  a.row = g.x;
  by_shape(a.d, bf16, [&](auto p, auto k) {
    constexpr int P = decltype(p)::value, K = decltype(k)::value;
    if (bf16) {
      if constexpr (P < 256 || K < 8)   // (8192 elements are 1024 vectors of eight)
        hipLaunchKernelGGL((pdssm_norm_kernel<SsBf16, P, K>), dim3(g.x, g.y), dim3(256), 0, st, a);
    } else {
      hipLaunchKernelGGL((pdssm_norm_kernel<SsF32, P, K>), dim3(g.x, g.y), dim3(256), 0, st, a);
    }
  });
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NmArgs& args, int bf16, hipStream_t st) {
  NmArgs a = args;
  const LaGrid g = la_grid_rows((long long)a.tiles * a.chunks, 256);
  a.row = g.x;
  by_shape(a.d, bf16, [&](auto p, auto k) {
    constexpr int P = decltype(p)::value, K = decltype(k)::value;
    if (bf16) {
      if constexpr (P < 256 || K < 8)
        hipLaunchKernelGGL((pdssm_norm_bwd_kernel<SsBf16, P, K>), dim3(g.x, g.y), dim3(256), 0, st, a);
    } else {
      hipLaunchKernelGGL((pdssm_norm_bwd_kernel<SsF32, P, K>), dim3(g.x, g.y), dim3(256), 0, st, a);
    }
  });
  return hipGetLastError();
}

}  // namespace pdscan
