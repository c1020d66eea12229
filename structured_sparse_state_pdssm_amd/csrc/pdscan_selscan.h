// Selective state-space scan: a diagonal state of N values for every channel d,
//
//   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,   y_t = (C_t . h_t + D x_t) silu(z_t),
//
// d_t = softplus(dt_t + bias).  Channels of a group share B and C.
//
// What bounds it.  The decay differs by channel and by state, so no matrix
// product forms it: every cell (t, d, n) costs an exponential (8 cycles of a
// SIMD for 64 lanes) and four multiplications or additions (4 each), 24 cycles
// run step by step.  Run so, a layer has too few chains to fill the card, so time is
// split too, without doing the exponentials twice: a wave takes some steps of
// a tile, keeps their decays a_t and drives d_t x_t B_t in registers while it
// forms its end state from zero, learns through LDS the state that enters its
// steps, and runs the recurrence again on the registers (one multiply-add more:
// 28 cycles).  Sequences that are too few even so are cut into segments, whose
// contributions a pass of their own forms first.
//
// Layout.  A lane holds S states of one channel; NS lanes hold a channel, a wave
// 64 / NS channels.
#pragma once

#include "pdscan_ssm.h"

namespace pdscan {

// Decays a[s] = 2^(A2[s] w), A2 = A log2 e.
template <int S>
__device__ __forceinline__ void ss_load_A(float (&A2)[S], const float* A, int64_t ch, int n0, int N, bool ok) {
#pragma unroll
  for (int s = 0; s < S; ++s) A2[s] = ok && n0 + s < N ? A[ch * N + n0 + s] * kLog2e : 0.0f;
}

template <int S>
__device__ __forceinline__ void ss_load_state(float (&h)[S], const float* p, int64_t at, int n0, int N, bool ok) {
#pragma unroll
  for (int s = 0; s < S; ++s) h[s] = p && ok && n0 + s < N ? p[at * N + n0 + s] : 0.0f;
}
template <int S>
__device__ __forceinline__ void ss_store_state(const float (&h)[S], float* p, int64_t at, int n0, int N, bool ok) {
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (ok && n0 + s < N) p[at * N + n0 + s] = h[s];
}

// S floats of this lane in an LDS or global array of [..][S / 4][64] vectors (S = 2: pairs).
template <int S>
__device__ __forceinline__ void ss_lane_put(float* p, const float (&h)[S], int lane) {
  constexpr int U = S < 4 ? S : 4;
#pragma unroll
  for (int i = 0; i < S / U; ++i) {
    SsVec<float, U> v;
#pragma unroll
    for (int j = 0; j < U; ++j) v.e[j] = h[i * U + j];
    *(SsVec<float, U>*)(p + (i * 64 + lane) * U) = v;
  }
}
template <int S>
__device__ __forceinline__ void ss_lane_get(float (&h)[S], const float* p, int lane) {
  constexpr int U = S < 4 ? S : 4;
#pragma unroll
  for (int i = 0; i < S / U; ++i) {
    const SsVec<float, U> v = *(const SsVec<float, U>*)(p + (i * 64 + lane) * U);
#pragma unroll
    for (int j = 0; j < U; ++j) h[i * U + j] = v.e[j];
  }
}
template <int S>
__device__ __forceinline__ void ss_row_get(float (&b)[S], const float* p) {
  constexpr int U = S < 4 ? S : 4;
#pragma unroll
  for (int i = 0; i < S / U; ++i) {
    const SsVec<float, U> v = *(const SsVec<float, U>*)(p + i * U);
#pragma unroll
    for (int j = 0; j < U; ++j) b[i * U + j] = v.e[j];
  }
}

struct SsUnit {
  int sid, g, c0, end;           // segment; group; first channel of the workgroup, end of its group
  int block;                     // channel block over all groups
};
__device__ __forceinline__ bool ss_unit(const SsArgs& a, int per, SsUnit& u) {
  const int K = a.D / a.G, nb = (K + per - 1) / per;
  const long long n = (long long)a.s.segs * a.G * nb, id = ss_near(ss_block(a.row), n);
  if (id >= n) return false;
  u.block = (int)(id % ((long long)a.G * nb));
  u.sid = (int)(id / ((long long)a.G * nb));
  u.g = u.block / nb;
  u.c0 = u.g * K + u.block % nb * per;
  u.end = (u.g + 1) * K;
  return true;
}

// The tile of a gradient at step t of segment s: tiles of different segments do not meet.
__device__ __forceinline__ int64_t ss_tile(const SsArgs& a, const SsSeg& s, int sid, int t) {
  const int per = (a.s.L + kSsBwdTile - 1) / kSsBwdTile;
  return (a.s.cu ? (int64_t)sid : (int64_t)s.b * per) + s.t0 / kSsBwdTile + t / kSsBwdTile;
}

// ---- prompts

template <typename T, int S, int NS, int TS>
__global__ __launch_bounds__(256) void pdssm_selscan_kernel(const SsArgs a) {
  constexpr int W = kSsTimeWaves, CW = 64 / NS, TT = W * TS, NP = S * NS;
  constexpr int V = TS * CW / 64, VB = TS * NP / 64;   // elements of a thread when a tile is staged
  using E = typename T::E;
  __shared__ __align__(16) float2 du[TT][CW];          // step, step times input
  __shared__ __align__(16) float Bs[TT][NP], Cs[TT][NP];
  __shared__ __align__(16) float ys[TT][CW];
  __shared__ __align__(16) float Es[W][S * 64], Ps[W][S * 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (ss_block(a.row) == 0 && tid < 2 && a.header) a.header[tid] = 0;
  SsUnit u;
  SsSeg s;
  if (!ss_unit(a, CW, u) || !ss_segment(a.s, u.sid, s)) return;
  const int c = lane % CW, q = lane / CW, ch = u.c0 + c;
  const bool ok = ch < u.end;
  float A2[S], H[S];
  ss_load_A(A2, a.A, ch, q * S, a.N, ok);
  if (s.first)
    ss_load_state(H, a.h0, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
  else
    ss_load_state(H, a.seg, (int64_t)u.sid * a.D + ch, q * S, a.N, ok);

  // this thread's part of a tile: V channels of one step, VB states of one step
  const int st = tid * V / CW, sc = tid * V % CW, bt = tid * VB / NP, bn = tid * VB % NP;
  const bool sok = u.c0 + sc < u.end, bok = bn < a.N;   // whole vectors: sizes are multiples of 8
  const int64_t row0 = s.t0;
  const int64_t xat = s.vb * a.x.sb + (row0 + st) * a.x.st + u.c0 + sc, dat = s.vb * a.dt.sb + (row0 + st) * a.dt.st + u.c0 + sc;
  const int64_t zat = s.vb * a.z.sb + (row0 + st) * a.z.st + u.c0 + sc, yat = s.vb * a.y.sb + (row0 + st) * a.y.st + u.c0 + sc;
  const int64_t Bat = s.vb * a.Bm.sb + u.g * a.Bm.sh + (row0 + bt) * a.Bm.st + bn, Cat = s.vb * a.Cm.sb + u.g * a.Cm.sh + (row0 + bt) * a.Cm.st + bn;
  float bias[V], skip[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = a.bias && sok ? a.bias[u.c0 + sc + v] : 0.0f;
    skip[v] = a.skip && sok ? a.skip[u.c0 + sc + v] : 0.0f;
  }
  const bool gated = a.z.p != nullptr;
  SsVec<E, V> xn = {}, dn = {}, zn = {};
  SsVec<E, VB> Bn = {}, Cn = {};
  auto fetch = [&](int t) {
    if (sok && t + st < s.len) {
      xn = ss_load<T, V>(a.x.p, xat + (int64_t)t * a.x.st);
      dn = ss_load<T, V>(a.dt.p, dat + (int64_t)t * a.dt.st);
      if (gated) zn = ss_load<T, V>(a.z.p, zat + (int64_t)t * a.z.st);
    }
    if (bok && t + bt < s.len) {
      Bn = ss_load<T, VB>(a.Bm.p, Bat + (int64_t)t * a.Bm.st);
      Cn = ss_load<T, VB>(a.Cm.p, Cat + (int64_t)t * a.Cm.st);
    }
  };
  fetch(0);
  for (int t0 = 0; t0 < s.len; t0 += TT) {
    // stage: steps behind the end have d = 0, which leaves the state as it is
    const bool live = sok && t0 + st < s.len, blive = bok && t0 + bt < s.len;
    const SsVec<E, V> xc = xn, zc = zn;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float raw = T::get(dn.e[v]) + bias[v];
      const float d = !live ? 0.0f : a.softplus ? ss_softplus_of(raw, ss_decay(raw)) : raw;
      du[st][sc + v] = make_float2(d, live ? d * T::get(xc.e[v]) : 0.0f);
    }
    {
      SsVec<float, VB> b, k;
#pragma unroll
      for (int v = 0; v < VB; ++v) {
        b.e[v] = blive ? T::get(Bn.e[v]) : 0.0f;
        k.e[v] = blive ? T::get(Cn.e[v]) : 0.0f;
      }
      *(SsVec<float, VB>*)&Bs[bt][bn] = b;
      *(SsVec<float, VB>*)&Cs[bt][bn] = k;
    }
    __syncthreads();
    if (t0 + TT < s.len) fetch(t0 + TT);

    // this wave's steps from zero
    float dec[TS][S], drv[TS][S], h[S], P[S], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < S; ++j) h[j] = 0.0f;
#pragma unroll
    for (int t = 0; t < TS; ++t) {
      const float2 w = du[wave * TS + t][c];
      float b[S];
      ss_row_get(b, &Bs[wave * TS + t][q * S]);
      sum += w.x;
#pragma unroll
      for (int j = 0; j < S; ++j) {
        dec[t][j] = ss_exp2(w.x * A2[j]);
        drv[t][j] = w.y * b[j];
        h[j] = __builtin_fmaf(dec[t][j], h[j], drv[t][j]);
      }
    }
#pragma unroll
    for (int j = 0; j < S; ++j) P[j] = ss_exp2(sum * A2[j]);
    ss_lane_put(Es[wave], h, lane);
    ss_lane_put(Ps[wave], P, lane);
    __syncthreads();
    // the state that enters them, and the one behind the tile
#pragma unroll
    for (int j = 0; j < S; ++j) h[j] = H[j];
#pragma unroll
    for (int v = 0; v < W; ++v) {
      float e[S], p[S];
      ss_lane_get(e, Es[v], lane);
      ss_lane_get(p, Ps[v], lane);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        if (v == wave) h[j] = H[j];
        H[j] = __builtin_fmaf(p[j], H[j], e[j]);
      }
    }
    // and the steps again
#pragma unroll
    for (int t4 = 0; t4 < TS; t4 += 4) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t4 + i;
        float k[S];
        ss_row_get(k, &Cs[wave * TS + t][q * S]);
        y[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < S; ++j) {
          h[j] = __builtin_fmaf(dec[t][j], h[j], drv[t][j]);
          y[i] = __builtin_fmaf(k[j], h[j], y[i]);
        }
      }
      // four steps' sums over the states, one step a row of 16 lanes
      float r = ss_fold_rows(y[0], y[1], y[2], y[3]);
      if constexpr (NS == 8) r += ss_dpp<kDppRor8>(r);
      if (NS == 4 || (lane & 15) < CW) ys[wave * TS + t4 + (lane >> 4)][lane & (CW - 1)] = r;
    }
    __syncthreads();
    if (live) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v] = __builtin_fmaf(skip[v], T::get(xc.e[v]), ys[st][sc + v]);
        if (gated) {
          const float z = T::get(zc.e[v]);
          o[v] *= z * ss_sigmoid(z);
        }
      }
      ss_store<T, V>(a.y.p, yat + (int64_t)t0 * a.y.st, o);
    }
  }
  if (s.last && wave == 0) ss_store_state(H, a.hL, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
}

// ---- contributions of segments
//
// The state that a segment adds, from zero, and the sum of its steps; a wave
// takes its channels through the segment alone.  With ckpt it also writes the
// state and the sum at the start of every tile of the gradient.  Backwards
// (REV) it is the adjoint state that flows out of the segment's start,
// l = a_t (l + g_t C_t), with g the gradient of y before its gate.
template <typename T, int S, int NS, bool REV>
__global__ __launch_bounds__(256) void pdssm_selscan_state_kernel(const SsArgs a) {
  constexpr int CG = kSsStateGroups, CW = 64 / NS, CC = CG * CW, NP = S * NS, TT = 16;
  constexpr int V = TT * CC / 256, VB = TT * NP / 64 < 8 ? TT * NP / 64 : 8, BT = TT * NP / VB;   // B by BT threads
  using E = typename T::E;
  __shared__ __align__(16) float2 du[2][TT][CC];
  __shared__ __align__(16) float Bs[2][TT][NP];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  SsUnit u;
  SsSeg s;
  if (!ss_unit(a, CC, u) || !ss_segment(a.s, u.sid, s)) return;
  if (REV ? s.first : (s.last && !a.ckpt)) return;   // nobody asks for it
  const int c = lane / NS, q = lane % NS, ch = u.c0 + wave * CW + c;
  const bool ok = ch < u.end;
  float A2[S], h[S];
  ss_load_A(A2, a.A, ch, q * S, a.N, ok);
#pragma unroll
  for (int j = 0; j < S; ++j) h[j] = 0.0f;
  const int st = tid * V / CC, sc = tid * V % CC, bt = tid * VB / NP, bn = tid * VB % NP;
  const bool sok = u.c0 + sc < u.end, bok = tid < BT && bn < a.N, gated = REV && a.z.p;
  const LaView &vx = REV ? a.gy : a.x, &vb = REV ? a.Cm : a.Bm;
  const int64_t row0 = s.t0;
  const int64_t xat = s.vb * vx.sb + (row0 + st) * vx.st + u.c0 + sc, dat = s.vb * a.dt.sb + (row0 + st) * a.dt.st + u.c0 + sc;
  const int64_t zat = s.vb * a.z.sb + (row0 + st) * a.z.st + u.c0 + sc, Bat = s.vb * vb.sb + u.g * vb.sh + (row0 + bt) * vb.st + bn;
  float bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) bias[v] = a.bias && sok ? a.bias[u.c0 + sc + v] : 0.0f;
  SsVec<E, V> xn = {}, dn = {}, zn = {};
  SsVec<E, VB> Bn = {};
  const int tiles = (s.len + TT - 1) / TT;
  auto fetch = [&](int t) {
    if (sok && t + st < s.len) {
      xn = ss_load<T, V>(vx.p, xat + (int64_t)t * vx.st);
      dn = ss_load<T, V>(a.dt.p, dat + (int64_t)t * a.dt.st);
      if (gated) zn = ss_load<T, V>(a.z.p, zat + (int64_t)t * a.z.st);
    }
    if (bok && t + bt < s.len) Bn = ss_load<T, VB>(vb.p, Bat + (int64_t)t * vb.st);
  };
  auto at = [&](int i) { return (REV ? tiles - 1 - i : i) * TT; };
  if (tiles) fetch(at(0));
  double total = 0.0;   // (long sums of steps: fp32 inside a tile)
  const int wblk = u.c0 % (a.D / a.G) / CW + wave;   // wave's channel block in its group
  const int nblk = (a.D / a.G + CW - 1) / CW;
  for (int i = 0; i < tiles; ++i) {
    const int t0 = at(i), p = i & 1;
    const bool live = sok && t0 + st < s.len, blive = bok && t0 + bt < s.len;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float raw = T::get(dn.e[v]) + bias[v];
      const float d = !live ? 0.0f : a.softplus ? ss_softplus_of(raw, ss_decay(raw)) : raw;
      float x = live ? T::get(xn.e[v]) : 0.0f;
      if (!REV) x = live ? d * x : 0.0f;
      if (gated && live) {
        const float z = T::get(zn.e[v]);
        x *= z * ss_sigmoid(z);
      }
      du[p][st][sc + v] = make_float2(d, x);
    }
    if (tid < BT) {
      SsVec<float, VB> b;
#pragma unroll
      for (int v = 0; v < VB; ++v) b.e[v] = blive ? T::get(Bn.e[v]) : 0.0f;
      *(SsVec<float, VB>*)&Bs[p][bt][bn] = b;
    }
    __syncthreads();
    if (i + 1 < tiles) fetch(at(i + 1));
    if (!REV && a.ckpt && t0 % kSsBwdTile == 0) {
      const int64_t tile = ss_tile(a, s, u.sid, t0);
      if (wblk < nblk) ss_lane_put(a.ckpt + ((tile * a.G + u.g) * nblk + wblk) * (S * 64), h, lane);
      if (ok && q == 0) a.cum[tile * a.D + ch] = (float)total;
    }
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < TT; ++k) {
      const int t = REV ? TT - 1 - k : k;
      const float2 w = du[p][t][wave * CW + c];
      float b[S];
      ss_row_get(b, &Bs[p][t][q * S]);
      sum += w.x;
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const float d = ss_exp2(w.x * A2[j]);
        h[j] = REV ? d * __builtin_fmaf(w.y, b[j], h[j]) : __builtin_fmaf(d, h[j], w.y * b[j]);
      }
    }
    total += (double)sum;
  }
  if (!a.seg) return;
  ss_store_state(h, REV ? a.adj : a.seg, (int64_t)u.sid * a.D + ch, q * S, a.N, ok);
  if (!REV && ok && q == 0) a.sum[(int64_t)u.sid * a.D + ch] = (float)total;
}

// ---- gradient
//
//   l_t = g_t C_t + a_{t+1} l_{t+1}                    g = g_y silu(z)
//   g_C = sum_d g h        g_B = sum_d l (d x)         g_x = g D + d (l . B)
//   g_d = x (l . B) + sum_n A q h_{t-1}                q = a_t l_t
//   g_A = sum_t d q h_{t-1}
//
// Tiles of 32 steps from the segment's end, each from the state at its start
// (written by the state pass): four waves take eight steps each, forwards and
// backwards from zero first, then, with what enters at both ends, again on the
// decays and states in registers.  Two such rows of waves, side by side in
// the channels, share a workgroup so that half as many partial sums of g_B and g_C are left.
template <typename T, int S, int NS>
__global__ __launch_bounds__(512) void pdssm_selscan_bwd_kernel(const SsArgs a) {
  constexpr int W = kSsTimeWaves, CG = kSsBwdGroups, TS = kSsBwdSteps, TT = W * TS, CW = 64 / NS, CC = CG * CW, NP = S * NS;
  constexpr int V = TT * CC / 512;
  constexpr int VB = TT * NP / 256 < 1 ? 1 : TT * NP / 256;   // B by the first four waves, C by the others
  using E = typename T::E;
  __shared__ __align__(16) float4 pre[TT][CC];     // d, d x, g
  __shared__ __align__(16) float Bs[TT][NP], Cs[TT][NP];
  __shared__ __align__(16) float outs[3][TT][CC];  // C . h, l . B, sum A q h
  __shared__ __align__(16) float gBs[CG][TT][NP], gCs[CG][TT][NP];
  __shared__ __align__(16) float Es[CG * W][S * 64], Ps[CG * W][S * 64], Rs[CG * W][S * 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = (tid >> 6) % W, cg = (tid >> 6) / W;
  if (ss_block(a.row) == 0 && tid < 2) a.header[tid] = 0;
  SsUnit u;
  if (!ss_unit(a, CC, u)) return;
  SsSeg s;
  const int c = lane / NS, q = lane % NS, ch = u.c0 + cg * CW + c;
  const bool ok = ch < u.end;
  const bool found = ss_segment(a.s, u.sid, s);
  if (!found || s.len <= 0) {   // no rows: nothing but sums of none and what passes through
    const float zero[S] = {};
    if (wave == 0) {
      ss_store_state(zero, a.partA, (int64_t)u.sid * a.D + ch, q * S, a.N, ok);
      if (ok && q < 2) a.partD[((int64_t)u.sid * 2 + q) * a.D + ch] = 0.0f;
      if (found && s.first && a.gh0) {
        float r[S];
        ss_load_state(r, a.ghL, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
        ss_store_state(r, a.gh0, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
      }
    }
    return;
  }
  float A2[S], An[S], R[S], H0[S], gA[S];
  ss_load_A(A2, a.A, ch, q * S, a.N, ok);
  ss_load_state(An, a.A, ch, q * S, a.N, ok);
  if (s.last)
    ss_load_state(R, a.ghL, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
  else
    ss_load_state(R, a.adj, (int64_t)u.sid * a.D + ch, q * S, a.N, ok);
  if (s.first)
    ss_load_state(H0, a.h0, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
  else
    ss_load_state(H0, a.seg, (int64_t)u.sid * a.D + ch, q * S, a.N, ok);
  const bool enters = !s.first || a.h0;
#pragma unroll
  for (int j = 0; j < S; ++j) gA[j] = 0.0f;

  const int st = tid * V / CC, sc = tid * V % CC;
  const int btid = tid & 255, bt = btid * VB / NP, bn = btid * VB % NP;
  const bool second = tid >= 256, sok = u.c0 + sc < u.end, bok = bt < TT && bn < a.N, gated = a.z.p != nullptr;
  const LaView& vbc = second ? a.Cm : a.Bm;
  const int64_t row0 = s.t0, r = row0 + st, cc = u.c0 + sc;
  const int64_t xat = s.vb * a.x.sb + r * a.x.st + cc, dat = s.vb * a.dt.sb + r * a.dt.st + cc, zat = s.vb * a.z.sb + r * a.z.st + cc;
  const int64_t gat = s.vb * a.gy.sb + r * a.gy.st + cc;
  const int64_t gxat = s.vb * a.gx.sb + r * a.gx.st + cc, gdat = s.vb * a.gdt.sb + r * a.gdt.st + cc, gzat = s.vb * a.gz.sb + r * a.gz.st + cc;
  const int64_t Bat = s.vb * vbc.sb + u.g * vbc.sh + (row0 + bt) * vbc.st + bn;
  float bias[V], skip[V], gD[V], gb[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = a.bias && sok ? a.bias[cc + v] : 0.0f;
    skip[v] = a.skip && sok ? a.skip[cc + v] : 0.0f;
    gD[v] = gb[v] = 0.0f;
  }
  const int wblk = u.c0 % (a.D / a.G) / CW + cg, nblk = (a.D / a.G + CW - 1) / CW;
  SsVec<E, V> xn = {}, dn = {}, zn = {}, gn = {};
  SsVec<E, VB> Bn = {};
  float hn[S], cumn = 0.0f;
  auto fetch = [&](int t) {
    if (sok && t + st < s.len) {
      xn = ss_load<T, V>(a.x.p, xat + (int64_t)t * a.x.st);
      dn = ss_load<T, V>(a.dt.p, dat + (int64_t)t * a.dt.st);
      gn = ss_load<T, V>(a.gy.p, gat + (int64_t)t * a.gy.st);
      if (gated) zn = ss_load<T, V>(a.z.p, zat + (int64_t)t * a.z.st);
    }
    if (bok && t + bt < s.len) Bn = ss_load<T, VB>(vbc.p, Bat + (int64_t)t * vbc.st);
    const int64_t tile = ss_tile(a, s, u.sid, t);
    if (wblk < nblk) ss_lane_get(hn, a.ckpt + ((tile * a.G + u.g) * nblk + wblk) * (S * 64), lane);
    cumn = ok ? a.cum[tile * a.D + ch] : 0.0f;
  };
#pragma unroll
  for (int j = 0; j < S; ++j) hn[j] = 0.0f;
  const int last = (s.len - 1) / TT * TT;
  fetch(last);
  for (int t0 = last; t0 >= 0; t0 -= TT) {
    const bool live = sok && t0 + st < s.len, blive = bok && t0 + bt < s.len;
    float x[V], d[V], g[V], sg[V], gz[V];   // input, step, gradient behind the gate, slope of the step, of the gate
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float raw = T::get(dn.e[v]) + bias[v], e = ss_decay(raw);
      x[v] = live ? T::get(xn.e[v]) : 0.0f;
      d[v] = !live ? 0.0f : a.softplus ? ss_softplus_of(raw, e) : raw;
      sg[v] = a.softplus ? ss_sigmoid_of(raw, e) : 1.0f;
      g[v] = live ? T::get(gn.e[v]) : 0.0f;
      gz[v] = 0.0f;
      if (gated && live) {
        const float z = T::get(zn.e[v]), k = ss_sigmoid(z);
        gz[v] = g[v] * k * __builtin_fmaf(z, 1.0f - k, 1.0f);
        g[v] *= z * k;
      }
      pre[st][sc + v] = make_float4(d[v], d[v] * x[v], g[v], 0.0f);
    }
    if (bt < TT) {
      SsVec<float, VB> b;
#pragma unroll
      for (int v = 0; v < VB; ++v) b.e[v] = blive ? T::get(Bn.e[v]) : 0.0f;
      *(SsVec<float, VB>*)(second ? &Cs[bt][bn] : &Bs[bt][bn]) = b;
    }
    float H[S];
#pragma unroll
    for (int j = 0; j < S; ++j) H[j] = enters ? __builtin_fmaf(ss_exp2(cumn * A2[j]), H0[j], hn[j]) : hn[j];
    __syncthreads();
    if (t0) fetch(t0 - TT);

    // from zero, forwards and backwards
    const int me = cg * W + wave, tw = wave * TS, lc = cg * CW + c;
    float dec[TS][S], hs[TS][S], h[S], l[S], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < S; ++j) h[j] = l[j] = 0.0f;
#pragma unroll
    for (int t = 0; t < TS; ++t) {
      const float4 w = pre[tw + t][lc];
      float b[S];
      ss_row_get(b, &Bs[tw + t][q * S]);
      sum += w.x;
#pragma unroll
      for (int j = 0; j < S; ++j) {
        dec[t][j] = ss_exp2(w.x * A2[j]);
        hs[t][j] = w.y * b[j];
        h[j] = __builtin_fmaf(dec[t][j], h[j], hs[t][j]);
      }
    }
    ss_lane_put(Es[me], h, lane);
#pragma unroll
    for (int j = 0; j < S; ++j) h[j] = ss_exp2(sum * A2[j]);
    ss_lane_put(Ps[me], h, lane);
#pragma unroll
    for (int t = TS - 1; t >= 0; --t) {
      const float g1 = pre[tw + t][lc].z;
      float k[S];
      ss_row_get(k, &Cs[tw + t][q * S]);
#pragma unroll
      for (int j = 0; j < S; ++j) l[j] = dec[t][j] * __builtin_fmaf(g1, k[j], l[j]);
    }
    ss_lane_put(Rs[me], l, lane);
    __syncthreads();
    // what enters at both ends of this wave's steps, and at the tile's start
#pragma unroll
    for (int j = 0; j < S; ++j) h[j] = H[j];
#pragma unroll
    for (int v = 0; v < W - 1; ++v) {
      float e[S], p[S];
      ss_lane_get(e, Es[cg * W + v], lane);
      ss_lane_get(p, Ps[cg * W + v], lane);
#pragma unroll
      for (int j = 0; j < S; ++j)
        if (v < wave) h[j] = __builtin_fmaf(p[j], h[j], e[j]);
    }
#pragma unroll
    for (int v = W - 1; v >= 0; --v) {
      float e[S], p[S];
      ss_lane_get(e, Rs[cg * W + v], lane);
      ss_lane_get(p, Ps[cg * W + v], lane);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        if (v == wave) l[j] = R[j];
        R[j] = __builtin_fmaf(p[j], R[j], e[j]);
      }
    }
    float hin[S];
#pragma unroll
    for (int j = 0; j < S; ++j) hin[j] = h[j];
#pragma unroll
    for (int t = 0; t < TS; ++t)
#pragma unroll
      for (int j = 0; j < S; ++j) hs[t][j] = h[j] = __builtin_fmaf(dec[t][j], h[j], hs[t][j]);
#pragma unroll
    for (int t4 = TS - 4; t4 >= 0; t4 -= 4) {
      float vB[4][S], vC[4][S];
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const int t = t4 + i;
        const float4 w = pre[tw + t][lc];
        float b[S], k[S], y = 0.0f, lb = 0.0f, pa = 0.0f;
        ss_row_get(b, &Bs[tw + t][q * S]);
        ss_row_get(k, &Cs[tw + t][q * S]);
#pragma unroll
        for (int j = 0; j < S; ++j) {
          l[j] = __builtin_fmaf(w.z, k[j], l[j]);
          vB[i][j] = w.y * l[j];
          vC[i][j] = w.z * hs[t][j];
          y = __builtin_fmaf(k[j], hs[t][j], y);
          lb = __builtin_fmaf(b[j], l[j], lb);
          l[j] *= dec[t][j];
          const float p = l[j] * (t ? hs[t ? t - 1 : 0][j] : hin[j]);
          pa = __builtin_fmaf(An[j], p, pa);
          gA[j] = __builtin_fmaf(w.x, p, gA[j]);
        }
        // over the states: lanes next to each other
        y += ss_dpp<kDppXor1>(y);
        lb += ss_dpp<kDppXor1>(lb);
        pa += ss_dpp<kDppXor1>(pa);
        y += ss_dpp<kDppXor2>(y);
        lb += ss_dpp<kDppXor2>(lb);
        pa += ss_dpp<kDppXor2>(pa);
        if constexpr (NS == 8) {
          y += ss_dpp<kDppHalfMirror>(y);
          lb += ss_dpp<kDppHalfMirror>(lb);
          pa += ss_dpp<kDppHalfMirror>(pa);
        }
        if (q < 3) outs[q][tw + t][lc] = q == 0 ? y : q == 1 ? lb : pa;
      }
      // over the channels: four steps' sums, one step a row of 16 lanes
      float rB[S], rC[S];
#pragma unroll
      for (int j = 0; j < S; ++j) {
        rB[j] = ss_fold_rows(vB[0][j], vB[1][j], vB[2][j], vB[3][j]);
        rC[j] = ss_fold_rows(vC[0][j], vC[1][j], vC[2][j], vC[3][j]);
        rB[j] += ss_dpp<kDppRor8>(rB[j]);
        rC[j] += ss_dpp<kDppRor8>(rC[j]);
        if constexpr (NS == 4) {
          rB[j] += ss_dpp<kDppRor4>(rB[j]);
          rC[j] += ss_dpp<kDppRor4>(rC[j]);
        }
      }
      if ((lane & 15) < NS) {
#pragma unroll
        for (int j = 0; j < S; ++j) {
          gBs[cg][tw + t4 + (lane >> 4)][q * S + j] = rB[j];
          gCs[cg][tw + t4 + (lane >> 4)][q * S + j] = rC[j];
        }
      }
    }
    __syncthreads();
    if (live) {
      float ox[V], od[V], oz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float y = outs[0][st][sc + v], lb = outs[1][st][sc + v], pa = outs[2][st][sc + v];
        ox[v] = __builtin_fmaf(d[v], lb, g[v] * skip[v]);
        od[v] = __builtin_fmaf(x[v], lb, pa) * sg[v];
        oz[v] = gz[v] * __builtin_fmaf(skip[v], x[v], y);
        gD[v] = __builtin_fmaf(g[v], x[v], gD[v]);
        gb[v] += od[v];
      }
      ss_store<T, V>(a.gx.p, gxat + (int64_t)t0 * a.gx.st, ox);
      ss_store<T, V>(a.gdt.p, gdat + (int64_t)t0 * a.gdt.st, od);
      if (gated) ss_store<T, V>(a.gz.p, gzat + (int64_t)t0 * a.gz.st, oz);
    }
    // this workgroup's part of g_B (first half of the threads) and g_C
    if (bt < TT && bn < a.N && t0 + bt < s.len) {
      const float(*src)[TT][NP] = second ? gCs : gBs;
      const int nb = a.G * ((a.D / a.G + CC - 1) / CC);
      const int64_t row = s.vb * a.s.L + s.t0 + t0 + bt;
      float* o = a.part + ((((int64_t)(second ? nb : 0) + u.block) * a.rows) + row) * a.N + bn;
      SsVec<float, VB> v;
#pragma unroll
      for (int j = 0; j < VB; ++j) v.e[j] = src[0][bt][bn + j] + src[1][bt][bn + j];
      *(SsVec<float, VB>*)o = v;
    }
  }
  if (s.first && wave == 0 && a.gh0) ss_store_state(R, a.gh0, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
  // sums over this workgroup's steps: the four waves', then the staging threads' of every channel
  __syncthreads();
  const int me = cg * W + wave;
  ss_lane_put(Es[me], gA, lane);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    outs[0][st][sc + v] = gD[v];
    outs[1][st][sc + v] = gb[v];
  }
  __syncthreads();
  if (wave == 0) {
    float sumA[S], e[S];
    ss_lane_get(sumA, Es[cg * W], lane);
    for (int v = 1; v < W; ++v) {
      ss_lane_get(e, Es[cg * W + v], lane);
#pragma unroll
      for (int j = 0; j < S; ++j) sumA[j] += e[j];
    }
    ss_store_state(sumA, a.partA, (int64_t)u.sid * a.D + ch, q * S, a.N, ok);
    if (ok && q < 2) {
      float o = 0.0f;
      for (int t = 0; t < TT; ++t) o += outs[q][t][cg * CW + c];
      a.partD[((int64_t)u.sid * 2 + q) * a.D + ch] = o;
    }
  }
}

// ---- one token
//
// Four states a lane, a channel in neighbouring lanes: the state streams
// through in whole lines, once each way, which is the time.
template <typename T, int NS>
__global__ __launch_bounds__(256) void pdssm_selscan_step_kernel(const SsStepArgs a) {
  constexpr int CW = 256 / NS;
  __shared__ int dup;
  const int tid = threadIdx.x, nb = (a.D + CW - 1) / CW;
  const unsigned id = ss_block(a.row);
  const int b = id / nb, ch = id % nb * CW + tid / NS, q = tid % NS, n0 = q * 4;
  if (b >= a.B) return;
  const int slot = a.idx ? a.idx[b] : b;
  const bool ok = ch < a.D;
  bool bad = slot < 0 || slot >= a.slots;
  if (!bad && a.idx) {
    // a slot named twice: the first row has it
    if (tid == 0) dup = 0;
    __syncthreads();
    int found = 0;
    for (int r = tid; r < b; r += 256) found |= a.idx[r] == slot;
    if (found) dup = 1;
    __syncthreads();
    bad = dup;
  }
  if (bad) {   // an empty row gives zeros; a slot past the pool, or another row's, NaN
    const float f = slot < 0 ? 0.0f : __builtin_nanf("");
    if (ok && q == 0) ss_store<T, 1>(a.y.p, (int64_t)b * a.y.sb + ch, &f);
    return;
  }
  if (!ok) return;   // (whole channels: their lanes leave together)
  const int g = ch / (a.D / a.G);
  const bool has = n0 < a.N;
  float4 h = make_float4(0, 0, 0, 0), A = h;
  float B[4] = {}, C[4] = {};
  float* hp = a.state + ((int64_t)slot * a.D + ch) * a.N + n0;
  if (has) {
    h = *(const float4*)hp;
    A = *(const float4*)(a.A + (int64_t)ch * a.N + n0);
    const auto vb = ss_load<T, 4>(a.Bm.p, (int64_t)b * a.Bm.sb + (int64_t)g * a.Bm.sh + n0);
    const auto vc = ss_load<T, 4>(a.Cm.p, (int64_t)b * a.Cm.sb + (int64_t)g * a.Cm.sh + n0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      B[i] = T::get(vb.e[i]);
      C[i] = T::get(vc.e[i]);
    }
  }
  const float x = T::get(((const typename T::E*)a.x.p)[(int64_t)b * a.x.sb + ch]);
  const float raw = T::get(((const typename T::E*)a.dt.p)[(int64_t)b * a.dt.sb + ch]) + (a.bias ? a.bias[ch] : 0.0f);
  const float d = a.softplus ? ss_softplus_of(raw, ss_decay(raw)) : raw, u = d * x, w = d * kLog2e;
  h.x = __builtin_fmaf(ss_exp2(w * A.x), h.x, u * B[0]);
  h.y = __builtin_fmaf(ss_exp2(w * A.y), h.y, u * B[1]);
  h.z = __builtin_fmaf(ss_exp2(w * A.z), h.z, u * B[2]);
  h.w = __builtin_fmaf(ss_exp2(w * A.w), h.w, u * B[3]);
  float y = (C[0] * h.x + C[1] * h.y) + (C[2] * h.z + C[3] * h.w);
  y += ss_dpp<kDppXor1>(y);
  if constexpr (NS >= 4) y += ss_dpp<kDppXor2>(y);
  if constexpr (NS >= 8) y += ss_dpp<kDppHalfMirror>(y);
  if constexpr (NS >= 16) y += ss_dpp<kDppRor8>(y);
  if (has) *(float4*)hp = h;
  if (q == 0) {
    y = __builtin_fmaf(a.skip ? a.skip[ch] : 0.0f, x, y);
    if (a.z.p) {
      const float z = T::get(((const typename T::E*)a.z.p)[(int64_t)b * a.z.sb + ch]);
      y *= z * ss_sigmoid(z);
    }
    ss_store<T, 1>(a.y.p, (int64_t)b * a.y.sb + ch, &y);
  }
}

}  // namespace pdscan
