// Short causal convolution of every channel with its own W taps:
//
//   y_t = act(bias + sum_j w_j x_{t-W+1+j}),  act(v) = v silu's sigmoid, or v.
//
// It reads and writes every cell once and is bound by that (12001 x 2048 in
// bf16, 23 sequences: 108 MB in 23 us, 4.7 TB/s).  A thread walks down 16 rows of 16
// bytes of channels, four of them under way, with the last W - 1 in registers.
// Backwards, with p the gradient before act (formed again from x):
//   g_x_t = sum_j w_j p_{t+W-1-j},  g_w_j = sum_t p_t x_{t-W+1+j}.
#include "pdscan_ssm.h"
#include "pdscan_ssm_launch.h"

namespace pdscan {

// Rows [t0, t1) of the sequence that row r belongs to (packed), its number in
// b; past the last sequence b = B, before the first -1.
struct CvSeq {
  int b, t0, t1;
};
__device__ __forceinline__ CvSeq cv_find(const CvArgs& a, int r) {
  int lo = 0, hi = a.B + 1;   // the first offset above r
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (a.cu[m] > r) hi = m;
    else lo = m + 1;
  }
  CvSeq s;
  s.b = lo - 1;
  s.t0 = s.b >= 0 ? a.cu[s.b] : 0;
  s.t1 = lo <= a.B ? a.cu[lo] : a.L;
  // offsets out of range are cut to it
  s.t0 = s.t0 < 0 ? 0 : s.t0;
  s.t1 = s.t1 > a.L ? a.L : s.t1;
  return s;
}
__device__ __forceinline__ CvSeq cv_seq(const CvArgs& a, int b) {
  CvSeq s;
  s.b = b;
  s.t0 = 0;
  s.t1 = a.L;
  if (a.cu) {
    s.t0 = a.cu[b];
    s.t1 = a.cu[b + 1];
    s.t0 = s.t0 < 0 ? 0 : s.t0 > a.L ? a.L : s.t0;
    s.t1 = s.t1 < s.t0 ? s.t0 : s.t1 > a.L ? a.L : s.t1;
  }
  return s;
}

// V channels of row r of sequence s, or of the state before it.
template <typename T, int W, int V>
__device__ __forceinline__ SsRaw<T, V> cv_row(const CvArgs& a, const CvSeq& s, int64_t vb, int r, int c) {
  SsRaw<T, V> x = {};
  const int i = W - 1 + r - s.t0;
  if (r >= s.t0)
    ss_load_raw(x, a.x.p, vb * a.x.sb + (int64_t)r * a.x.st + c);
  else if (a.x0 && i >= 0)
    ss_load_raw(x, a.x0, ((int64_t)s.b * (W - 1) + i) * a.D + c);
  return x;
}

template <int W, int V>
__device__ __forceinline__ void cv_weights(float (&w)[W][V], float (&bias)[V], const float* wp, const float* bp, int c) {
  constexpr int U = 4;   // (c is a multiple of it)
#pragma unroll
  for (int i = 0; i < V * W; i += U) {
    const auto x = ss_load<SsF32, U>(wp, (int64_t)c * W + i);
#pragma unroll
    for (int k = 0; k < U; ++k) w[(i + k) % W][(i + k) / W] = x.e[k];
  }
#pragma unroll
  for (int v = 0; v < V; v += U) {
    SsVec<float, U> x = {};
    if (bp) x = ss_load<SsF32, U>(bp, c + v);
#pragma unroll
    for (int k = 0; k < U; ++k) bias[v + k] = x.e[k];
  }
}

// y of the last row of win, whose rows end at the current one.
template <typename T, int W, int V>
__device__ __forceinline__ float cv_pre(const SsRaw<T, V>* win, const float (&w)[W][V], float bias, int v) {
  float p = bias;
#pragma unroll
  for (int j = 0; j < W; ++j) p = __builtin_fmaf(w[j][v], win[j].get(v), p);
  return p;
}

template <typename T, int W>
__global__ __launch_bounds__(256) void pdssm_conv_kernel(const CvArgs a) {
  constexpr int V = 16 / sizeof(typename T::E), U = 4;   // rows under way
  const int nv = a.D / V;
  unsigned id = ss_block(a.row) * 256 + threadIdx.x;   // (the host keeps threads below 2^31)
  if (id >= a.units) {
    // the state behind every sequence: its last rows, or what is left of the state before it
    id -= a.units;
    const int c = (int)(id % nv) * V;
    id /= nv;
    const int j = (int)(id % (W - 1));
    const int64_t b = id / (W - 1);
    if (b >= a.B) return;
    const CvSeq s = cv_seq(a, (int)b);
    ss_store_raw(a.xL, (b * (W - 1) + j) * a.D + c, cv_row<T, W, V>(a, s, a.cu ? 0 : b, s.t1 - (W - 1) + j, c));
    return;
  }
  const int c = (int)(id % nv) * V;
  const unsigned strip = id / nv;
  const int64_t vb = a.cu ? 0 : strip / a.strips;
  int r = (int)(strip % a.strips) * kCvRows;
  const int end = a.L - r < kCvRows ? a.L : r + kCvRows;
  float w[W][V], bias[V];
  cv_weights(w, bias, a.w, a.bias, c);
  while (r < end) {
    CvSeq s;
    if (a.cu)
      s = cv_find(a, r);
    else
      s = CvSeq{(int)vb, 0, a.L};
    if (s.b >= a.B) return;
    const int e = s.t1 < end ? s.t1 : end;
    if (e <= r) return;   // offsets out of order
    if (s.b < 0) {
      r = e;
      continue;
    }
    SsRaw<T, V> win[W - 1 + U];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = cv_row<T, W, V>(a, s, vb, r - (W - 1) + j, c);
    int64_t xp = vb * a.x.sb + (int64_t)r * a.x.st + c;
    int64_t yp = vb * a.y.sb + (int64_t)r * a.y.st + c;
    for (; r < e; r += U) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (r + i < e) ss_load_raw(win[W - 1 + i], a.x.p, xp + i * a.x.st);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (r + i >= e) break;
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float p = cv_pre<T, W, V>(win + i, w, bias[v], v);
          o[v] = a.silu ? p * ss_sigmoid<T>(p) : p;
        }
        ss_store<T, V>(a.y.p, yp + i * a.y.st, o);
      }
      xp += U * a.x.st;
      yp += U * a.y.st;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) win[j] = win[j + U];
    }
    r = e;
  }
}

// p of one row: the gradient before act, V channels.
template <typename T, int W, int V>
__device__ __forceinline__ void cv_grad(float (&p)[V], const SsRaw<T, V>* win, const SsRaw<T, V>& gy,
                                        const float (&w)[W][V], const float (&bias)[V], int silu) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float x = cv_pre<T, W, V>(win, w, bias[v], v);
    p[v] = gy.get(v);
    if (silu) {
      const float k = ss_sigmoid<T>(x);
      p[v] *= k * __builtin_fmaf(x, 1.0f - k, 1.0f);
    }
  }
}

// 64 columns of four channels, four strips of 32 rows each; a strip looks W - 1
// rows past its end.  The strips' sums of g_w and g_bias meet in LDS.  16 x 2048
// x 768 in bf16: 37 us, 169 MB at 4.6 TB/s, beside 33 us of the vector units; the
// call with its sums 41 us, with strips of 16 rows 47, of 64 54.
template <typename T, int W>
__global__ __launch_bounds__(256) void pdssm_conv_bwd_kernel(const CvArgs a) {
  constexpr int V = 4;
  __shared__ float red[kCvBwdStrips - 1][(W + 1) * V][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tiles = (a.D + 64 * V - 1) / (64 * V);
  const unsigned id = ss_block(a.row);
  if (id == 0 && threadIdx.x < 2) a.header[threadIdx.x] = 0;
  const int part = id / tiles, c = (id % tiles * 64 + lane) * V;
  if (part >= a.parts) return;
  const unsigned strip = (unsigned)part * kCvBwdStrips + wave;
  const int64_t vb = a.cu ? 0 : strip / a.strips;
  const bool has = c < a.D && vb < (a.cu ? 1 : a.B) && strip < (a.cu ? (unsigned)a.strips : (unsigned)a.B * a.strips);
  float gw[W][V] = {}, gb[V] = {};
  if (has) {
    int r = (int)(strip % a.strips) * kCvBwdRows;
    const int end = a.L - r < kCvBwdRows ? a.L : r + kCvBwdRows;
    float w[W][V], bias[V];
    cv_weights(w, bias, a.w, a.bias, c);
    while (r < end) {
      CvSeq s;
      if (a.cu)
        s = cv_find(a, r);
      else
        s = CvSeq{(int)vb, 0, a.L};
      if (s.b >= a.B) break;
      const int e = s.t1 < end ? s.t1 : end;
      if (e <= r) break;   // offsets out of order
      if (s.b < 0) {
        r = e;
        continue;
      }
      // win: rows t - W + 1 .. t + U - 1 of x; gp: p of the last W rows
      constexpr int U = 4;
      SsRaw<T, V> win[W - 1 + U] = {}, gy[U] = {};
      float gp[W][V] = {};
#pragma unroll
      for (int j = 0; j < W - 1; ++j) win[j] = cv_row<T, W, V>(a, s, vb, r - (W - 1) + j, c);
      int64_t xp = vb * a.x.sb + (int64_t)r * a.x.st + c, gyp = vb * a.gy.sb + (int64_t)r * a.gy.st + c;
      int64_t gxp = vb * a.gx.sb + (int64_t)(r - (W - 1)) * a.gx.st + c;
      const int stop = e + W - 1;
      for (int t0 = r; t0 < stop; t0 += U) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (t0 + i < s.t1 && t0 + i < stop) {
            ss_load_raw(win[W - 1 + i], a.x.p, xp + i * a.x.st);
            ss_load_raw(gy[i], a.gy.p, gyp + i * a.gy.st);
          }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int t = t0 + i;
          if (t >= stop) break;
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) gp[j][v] = gp[j + 1][v];
          if (t < s.t1) {
            cv_grad<T, W, V>(gp[W - 1], win + i, gy[i], w, bias, a.silu);
          } else {
#pragma unroll
            for (int v = 0; v < V; ++v) gp[W - 1][v] = 0.0f;
          }
          if (t < e) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
              for (int j = 0; j < W; ++j) gw[j][v] = __builtin_fmaf(gp[W - 1][v], win[i + j].get(v), gw[j][v]);
              gb[v] += gp[W - 1][v];
            }
          }
          const int to = t - (W - 1);
          if (to >= r) {
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
              o[v] = 0.0f;
#pragma unroll
              for (int j = 0; j < W; ++j) o[v] = __builtin_fmaf(w[j][v], gp[W - 1 - j][v], o[v]);
            }
            const int k = to - (s.t1 - (W - 1));
            if (k >= 0 && a.gxL) {   // one of the last rows: they are the state behind the sequence too
              const auto g = ss_load<T, V>(a.gxL, ((int64_t)s.b * (W - 1) + k) * a.D + c);
#pragma unroll
              for (int v = 0; v < V; ++v) o[v] += T::get(g.e[v]);
            }
            ss_store<T, V>(a.gx.p, gxp + i * a.gx.st, o);
          }
        }
        xp += U * a.x.st;
        gyp += U * a.gy.st;
        gxp += U * a.gx.st;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j] = win[j + U];
      }
      r = e;
    }
  }
  if (wave) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < W; ++j) red[wave - 1][v * W + j][lane] = gw[j][v];
      red[wave - 1][V * W + v][lane] = gb[v];
    }
  }
  __syncthreads();
  if (wave || c >= a.D) return;
  float* o = a.part + (int64_t)part * a.D * (W + 1);
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < W; ++j)
      o[(int64_t)(c + v) * W + j] = (gw[j][v] + red[0][v * W + j][lane]) + (red[1][v * W + j][lane] + red[2][v * W + j][lane]);
    o[(int64_t)a.D * W + c + v] = (gb[v] + red[0][V * W + v][lane]) + (red[1][V * W + v][lane] + red[2][V * W + v][lane]);
  }
}

// Gradient of the state before every sequence: what its first rows, and the
// state behind it where it is shorter than the window, have of it.
template <typename T, int W>
__global__ __launch_bounds__(256) void pdssm_conv_state_bwd_kernel(const CvArgs a) {
  constexpr int V = 4;
  const int nv = a.D / V;
  const unsigned id = ss_block(a.row) * 256 + threadIdx.x;
  const int c = (int)(id % nv) * V;
  const int64_t b = id / nv;
  if (b >= a.B) return;
  const CvSeq s = cv_seq(a, (int)b);
  const int64_t vb = a.cu ? 0 : b;
  const int len = s.t1 - s.t0;
  float w[W][V], bias[V], gp[W - 1][V];
  cv_weights(w, bias, a.w, a.bias, c);
#pragma unroll
  for (int t = 0; t < W - 1; ++t) {
    if (t < len) {
      SsRaw<T, V> win[W], gy;
#pragma unroll
      for (int j = 0; j < W; ++j) win[j] = cv_row<T, W, V>(a, s, vb, s.t0 + t - (W - 1) + j, c);
      ss_load_raw(gy, a.gy.p, vb * a.gy.sb + (int64_t)(s.t0 + t) * a.gy.st + c);
      cv_grad<T, W, V>(gp[t], win, gy, w, bias, a.silu);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) gp[t][v] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      o[v] = 0.0f;
#pragma unroll
      for (int j = 0; j <= i; ++j) o[v] = __builtin_fmaf(w[j][v], gp[i - j][v], o[v]);
    }
    if (a.gxL && i >= len) {
      const auto g = ss_load<T, V>(a.gxL, (b * (W - 1) + i - len) * a.D + c);
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] += T::get(g.e[v]);
    }
    ss_store<T, V>(a.gx0, (b * (W - 1) + i) * a.D + c, o);
  }
}

// One token of every row on a pool of states, which moves up one row in place.
template <typename T, int W>
__global__ __launch_bounds__(256) void pdssm_conv_step_kernel(const CvStepArgs a) {
  constexpr int V = 4;
  const int tid = threadIdx.x, nb = (a.D / V + 255) / 256;
  const unsigned id = ss_block(a.row);
  const int b = id / nb, c = (id % nb * 256 + tid) * V;
  if (b >= a.B) return;
  const int slot = a.idx ? a.idx[b] : b;
  const bool ok = c < a.D, has = ok && slot >= 0 && slot < a.slots;
  const int64_t yp = (int64_t)b * a.y.sb + c, sp = (int64_t)slot * (W - 1) * a.D + c;
  SsRaw<T, V> win[W] = {};
  float w[W][V] = {}, bias[V] = {}, o[V];
  if (has) {   // under way before the search for an earlier row of the same slot
#pragma unroll
    for (int j = 0; j < W - 1; ++j) ss_load_raw(win[j], a.state, sp + (int64_t)j * a.D);
    ss_load_raw(win[W - 1], a.x.p, (int64_t)b * a.x.sb + c);
    cv_weights(w, bias, a.w, a.bias, c);
  }
  if (ss_taken(a.idx, b, slot, a.slots, tid & 63)) {
    const float f = slot < 0 ? 0.0f : __builtin_nanf("");
    const float e[V] = {f, f, f, f};
    if (ok) ss_store<T, V>(a.y.p, yp, e);
    return;
  }
  if (!ok) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float p = cv_pre<T, W, V>(win, w, bias[v], v);
    o[v] = a.silu ? p * ss_sigmoid<T>(p) : p;
  }
  ss_store<T, V>(a.y.p, yp, o);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) ss_store_raw(a.state, sp + (int64_t)j * a.D, win[j + 1]);
}

#define PDSCAN_CONV(kernel, grid)                                                                            \
  do {                                                                                                       \
    const LaGrid g = grid;                                                                                   \
    a.row = g.x;                                                                                             \
    if (bf16) {                                                                                              \
      if (a.W == 2) hipLaunchKernelGGL((kernel<SsBf16, 2>), dim3(g.x, g.y), dim3(256), 0, st, a);             \
      else if (a.W == 3) hipLaunchKernelGGL((kernel<SsBf16, 3>), dim3(g.x, g.y), dim3(256), 0, st, a);        \
      else hipLaunchKernelGGL((kernel<SsBf16, 4>), dim3(g.x, g.y), dim3(256), 0, st, a);                      \
    } else {                                                                                                 \
      if (a.W == 2) hipLaunchKernelGGL((kernel<SsF32, 2>), dim3(g.x, g.y), dim3(256), 0, st, a);              \
      else if (a.W == 3) hipLaunchKernelGGL((kernel<SsF32, 3>), dim3(g.x, g.y), dim3(256), 0, st, a);         \
      else hipLaunchKernelGGL((kernel<SsF32, 4>), dim3(g.x, g.y), dim3(256), 0, st, a);                       \
    }                                                                                                        \
  } while (0)

hipError_t launch_conv_fwd(const CvArgs& args, int bf16, hipStream_t st) {
  CvArgs a = args;
  const int nv = a.D / (bf16 ? 8 : 4);
  a.units = (unsigned)cv_units(a, bf16);
  PDSCAN_CONV(pdssm_conv_kernel, la_grid_rows((a.units + (long long)a.B * (a.W - 1) * nv + 255) / 256, 256));
  return hipGetLastError();
}

hipError_t launch_conv_bwd(const CvArgs& args, int bf16, hipStream_t st) {
  CvArgs a = args;
  PDSCAN_CONV(pdssm_conv_bwd_kernel, la_grid_rows((long long)a.parts * ((a.D + 255) / 256), 256));
  if (a.gx0) PDSCAN_CONV(pdssm_conv_state_bwd_kernel, la_grid_rows(((long long)a.B * (a.D / 4) + 255) / 256, 256));
  return hipGetLastError();
}

hipError_t launch_conv_step(const CvStepArgs& args, int bf16, hipStream_t st) {
  CvStepArgs a = args;
  PDSCAN_CONV(pdssm_conv_step_kernel, la_grid_rows((long long)a.B * ((a.D / 4 + 255) / 256), 256));
  return hipGetLastError();
}

}  // namespace pdscan
