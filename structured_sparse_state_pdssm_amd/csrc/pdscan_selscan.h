// Selective state-space scan: a diagonal state of N values for every channel d,
//
//   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,   y_t = (C_t . h_t + D x_t) silu(z_t),
//
// d_t = softplus(dt_t + bias).  Channels of a group share B and C.
//
// What bounds it.  The decay differs by channel and by state, so no matrix
// product forms it: every cell (t, d, n) costs an exponential (8 cycles of a
// SIMD for 64 lanes; the exponential and the other units do not overlap) and four
// multiplications or additions (4 each), 24 cycles run step by step.  Run so, a
// layer has too few chains to fill the card, so time is split too, without
// doing the exponentials twice: a wave takes eight steps of a tile of 32,
// keeps their decays a_t and drives d_t x_t B_t in registers while it forms its
// end state from zero, learns through LDS the state that enters its steps, and
// runs the recurrence again on the registers (one multiply-add more: 28 cycles).
// Sequences that are too few even so are cut into runs, which start from
// states that a pass of its own forms first (ss_split).
//
// 16 x 2048 steps, 768 channels, 16 states, bf16: 141 us (159 under the
// profiler).  The vector units are what it waits for: 136 us at 2.1 GHz by their counter, of
// which the cells' 28 cycles are 84; the rest is what a (t, d) needs once (softplus, the gate,
// roundings) and the exchanges.  Memory, 205 MB, would take 40.  Three barriers a tile took 151, two 141.
// A tile's first wave could run its steps once, from the state that it knows, and its last
// one without an end state from zero: 134 us, the gradient 509 instead of 529.  But the state from
// tile to tile then takes an exponential's error at every step, not at every
// eighth (h_L after 77 steps off by 2.8e-7 instead of 1.3e-7); not done.
//
// Layout.  A lane holds S states of one channel; NS lanes hold a channel, a wave
// 64 / NS channels: four states a lane up to 32 (eight, and half the lanes,
// need twice the registers: 4 x 2048 x 768 of 32 states took 144 us forwards and
// 423 backwards when 116 and 350 were taken so, now 116 and 330).
#pragma once

#include "pdscan_ssm.h"

namespace pdscan {

// Decays a[s] = 2^(A2[s] w), A2 = A log2 e.
template <int S>
__device__ __forceinline__ void ss_load_A(float (&A2)[S], const float* A, int64_t ch, int n0, int N, bool ok) {
#pragma unroll
  for (int s = 0; s < S; ++s) A2[s] = ok && n0 + s < N ? ss_held_decay(A[ch * N + n0 + s] * kLog2e) : 0.0f;
}

// A lane's S states from the n0-th of channel row `at` (N is a multiple of 8: all of them or none).
template <int S>
__device__ __forceinline__ void ss_load_state(float (&h)[S], const float* p, int64_t at, int n0, int N, bool ok) {
  SsVec<float, S> v = {};
  if (p && ok && n0 < N) v = *(const SsVec<float, S>*)(p + at * N + n0);
#pragma unroll
  for (int s = 0; s < S; ++s) h[s] = v.e[s];
}
template <int S>
__device__ __forceinline__ void ss_store_state(const float (&h)[S], float* p, int64_t at, int n0, int N, bool ok) {
  SsVec<float, S> v;
#pragma unroll
  for (int s = 0; s < S; ++s) v.e[s] = h[s];
  if (ok && n0 < N) *(SsVec<float, S>*)(p + at * N + n0) = v;
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

// The first piece of the run that segment s is, counted over all.
__device__ __forceinline__ int ss_piece(const SsArgs& a, const SsSeg& s, int sid) {
  if (!a.s.cu) return __builtin_amdgcn_readfirstlane(s.b * a.npiece + s.t0 / a.piece);
  if (!a.pieces) return s.b;
  const int first = __builtin_amdgcn_readfirstlane(a.pieces[s.b]);
  return ss_piece_at(first, a.runs ? __builtin_amdgcn_readfirstlane(sid - a.runs[s.b]) * a.run : 0, a.npieces);
}
__device__ __forceinline__ int64_t ss_tile(const SsArgs& a, int b, int at, int t0, int t) {
  return ss_tile_of(a.s.cu ? 0 : (a.s.L + kSsBwdTile - 1) / kSsBwdTile, b, at, t0, t, kSsBwdTile);
}

// ---- prompts

template <typename T, int S, int NS, int TS>
__global__ __launch_bounds__(256, S >= 8 ? 2 : 3) void pdssm_selscan_kernel(const SsArgs a) {
  constexpr int W = kSsTimeWaves, CW = 64 / NS, TT = W * TS, NP = S * NS;
  constexpr int V = TS * CW / 64, VB = TS * NP / 64;   // elements of a thread when a tile is staged
  __shared__ __align__(16) float2 du2[2][TT][CW];      // step, step times input; of two tiles in turn
  __shared__ __align__(16) float Bs2[2][TT][NP], Cs2[2][TT][NP];
  __shared__ __align__(16) float ys[TT][CW], pars[2][CW];
  __shared__ __align__(16) float Es[W - 1][S * 64], Ps[W - 1][S * 64], Hs[2][S * 64];   // Hs: the state that enters a tile
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (ss_block(a.row) == 0 && tid < 2 && a.header) a.header[tid] = 0;
  SsUnit u;
  SsSeg s;
  if (!ss_unit(a, CW, u) || !ss_segment(a.s, u.sid, s)) return;
  const int c = lane % CW, q = lane / CW, ch = u.c0 + c;
  const bool ok = ch < u.end;
  float A2[S];
  ss_load_A(A2, a.A, ch, q * S, a.N, ok);
  if (wave == W - 1) {
    float H[S];
    if (a.seg)
      ss_load_state(H, a.seg, (int64_t)ss_piece(a, s, u.sid) * a.D + ch, q * S, a.N, ok);
    else
      ss_load_state(H, a.h0, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
    ss_lane_put(Hs[0], H, lane);
  }

  // this thread's part of a tile: V channels of one step, VB states of one step
  const int st = tid * V / CW, sc = tid * V % CW, bt = tid * VB / NP, bn = tid * VB % NP;
  const bool sok = u.c0 + sc < u.end, bok = bn < a.N;   // whole vectors: sizes are multiples of 8
  const uint32_t xo = ss_off<T>(a.x, st, sc), dto = ss_off<T>(a.dt, st, sc), zo = ss_off<T>(a.z, st, sc), yo = ss_off<T>(a.y, st, sc);
  const uint32_t Bo = ss_off<T>(a.Bm, bt, bn), Co = ss_off<T>(a.Cm, bt, bn);
  if (tid < CW) {
    pars[0][tid] = a.bias && ok ? a.bias[ch] : 0.0f;
    pars[1][tid] = a.skip && ok ? a.skip[ch] : 0.0f;
  }
  __syncthreads();
  const bool gated = a.z.p != nullptr;
  SsRaw<T, V> xn = {}, dn = {}, zn = {};
  SsRaw<T, VB> Bn = {}, Cn = {};
  const char *xp = ss_tile_at<T>(a.x, s.vb, s.t0, u.c0), *dp = ss_tile_at<T>(a.dt, s.vb, s.t0, u.c0), *zp = ss_tile_at<T>(a.z, s.vb, s.t0, u.c0);
  const char *Bp = ss_tile_at<T>(a.Bm, s.vb, s.t0, u.g * a.Bm.sh), *Cp = ss_tile_at<T>(a.Cm, s.vb, s.t0, u.g * a.Cm.sh);
  char* yp = ss_tile_at<T>(a.y, s.vb, s.t0, u.c0);
  auto fetch = [&](int t) {   // and the pointers on to the tile behind it
    if (sok && t + st < s.len) {
      ss_load_at(xn, xp, xo);
      ss_load_at(dn, dp, dto);
      if (gated) ss_load_at(zn, zp, zo);
    }
    if (bok && t + bt < s.len) {
      ss_load_at(Bn, Bp, Bo);
      ss_load_at(Cn, Cp, Co);
    }
    xp += ss_rows<T>(a.x, TT);
    dp += ss_rows<T>(a.dt, TT);
    zp += ss_rows<T>(a.z, TT);
    Bp += ss_rows<T>(a.Bm, TT);
    Cp += ss_rows<T>(a.Cm, TT);
  };
  fetch(0);
  // The outputs of a tile leave after the next one is staged: two barriers a tile.
  SsRaw<T, V> xc = {}, zc = {};
  auto finish = [&](bool live) {
    if (live) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = __builtin_fmaf(pars[1][sc + v], xc.get(v), ys[st][sc + v]);
      if (gated) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float z = zc.get(v);
          o[v] *= z * ss_sigmoid<T>(z);
        }
      }
      ss_store_at<T, V>(yp, yo, o);
    }
    yp += ss_rows<T>(a.y, TT);
  };
  int turn = 0;
  for (int t0 = 0; t0 < s.len; t0 += TT, turn ^= 1) {
    auto& du = du2[turn];
    auto& Bs = Bs2[turn];
    auto& Cs = Cs2[turn];
    // stage: steps behind the end have d = 0, which leaves the state as it is
    const bool live = sok && t0 + st < s.len;
    float d[V], none[V];
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = dn.get(v) + pars[0][sc + v];
    ss_steps<V, false>(d, none, a.softplus, live);
#pragma unroll
    for (int v = 0; v < V; ++v) du[st][sc + v] = make_float2(d[v], d[v] * xn.get(v));
    {   // (behind the end: of an earlier tile, with a step of zero)
      SsVec<float, VB> b, k;
#pragma unroll
      for (int v = 0; v < VB; ++v) {
        b.e[v] = Bn.get(v);
        k.e[v] = Cn.get(v);
      }
      *(SsVec<float, VB>*)&Bs[bt][bn] = b;
      *(SsVec<float, VB>*)&Cs[bt][bn] = k;
    }
    __syncthreads();
    if (t0) finish(sok);   // (a tile behind which there is another is whole)
    xc = xn;
    zc = zn;
    if (t0 + TT < s.len) fetch(t0 + TT);

    // this wave's steps from zero
    float dec[TS][S], drv[TS][S], h[S], P[S], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < S; ++j) h[j] = 0.0f;
#pragma unroll
    for (int t4 = 0; t4 < TS; t4 += 4) {
      float2 w[4];
      float b[4][S];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = du[wave * TS + t4 + i][c];
        ss_row_get(b[i], &Bs[wave * TS + t4 + i][q * S]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t4 + i;
        sum += w[i].x;
#pragma unroll
        for (int j = 0; j < S; ++j) {
          dec[t][j] = ss_exp2(w[i].x * A2[j]);
          drv[t][j] = w[i].y * b[i][j];
          h[j] = __builtin_fmaf(dec[t][j], h[j], drv[t][j]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    sum = ss_held_sum(sum);
#pragma unroll
    for (int j = 0; j < S; ++j) P[j] = ss_exp2(sum * A2[j]);
    if (wave < W - 1) {
      ss_lane_put(Es[wave], h, lane);
      ss_lane_put(Ps[wave], P, lane);
    }
    __syncthreads();
    // the state that enters them; the last wave's is behind the tile then
    float own[S];
#pragma unroll
    for (int j = 0; j < S; ++j) own[j] = h[j];
    ss_lane_get(h, Hs[turn], lane);
#pragma unroll
    for (int v = 0; v < W - 1; ++v) {
      if (v < wave) {
        float e[S], p[S];
        ss_lane_get(e, Es[v], lane);
        ss_lane_get(p, Ps[v], lane);
#pragma unroll
        for (int j = 0; j < S; ++j) h[j] = __builtin_fmaf(p[j], h[j], e[j]);
      }
    }
    if (wave == W - 1) {
#pragma unroll
      for (int j = 0; j < S; ++j) own[j] = __builtin_fmaf(P[j], h[j], own[j]);
      ss_lane_put(Hs[turn ^ 1], own, lane);
    }
    // and the steps again
#pragma unroll
    for (int t4 = 0; t4 < TS; t4 += 4) {
      float y[4], k[4][S];
#pragma unroll
      for (int i = 0; i < 4; ++i) ss_row_get(k[i], &Cs[wave * TS + t4 + i][q * S]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t4 + i;
        y[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < S; ++j) {
          h[j] = __builtin_fmaf(dec[t][j], h[j], drv[t][j]);
          y[i] = __builtin_fmaf(k[i][j], h[j], y[i]);
        }
      }
      // four steps' sums over the states, one step a row of 16 lanes
      float r = ss_fold_rows(y[0], y[1], y[2], y[3]);
      if constexpr (NS == 8) r += ss_dpp<kDppRor8>(r);
      if (NS == 4 || (lane & 15) < CW) ys[wave * TS + t4 + (lane >> 4)][lane & (CW - 1)] = r;
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __syncthreads();
  if (s.len > 0) finish(sok && (s.len - 1) / TT * TT + st < s.len);
  if (s.last && wave == W - 1) {
    float H[S];
    ss_lane_get(H, Hs[turn], lane);
    ss_store_state(H, a.hL, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
  }
}

// ---- contributions of pieces
//
// The state that a piece adds, from zero, and the sum of its steps; a wave
// takes its channels through the piece alone (16 x 2048 x 768 x 16
// 94 to 99 us under the profiler, 82 of them the vector units).  With ckpt it also writes the
// state and the sum at the start of every tile of the gradient.  Backwards
// (REV) it is the adjoint state that flows out of the piece's start,
// l = a_t (l + g_t C_t), with g the gradient of y before its gate.
template <int S, int NS>
struct SsStateLds {
  static constexpr int TT = 16, CC = kSsStateGroups * (64 / NS);
  alignas(16) float2 du[2][TT][CC];
  alignas(16) float Bs[2][TT][S * NS];
};
template <typename T, int S, int NS, bool REV>
__device__ __forceinline__ void ss_state_body(const SsArgs& a, SsStateLds<S, NS>& lds) {
  constexpr int CG = kSsStateGroups, CW = 64 / NS, CC = CG * CW, NP = S * NS, TT = 16;
  constexpr int V = TT * CC / 256, VB = TT * NP / 64 < 8 ? TT * NP / 64 : 8, BT = TT * NP / VB;   // B by BT threads
  auto& du = lds.du;
  auto& Bs = lds.Bs;
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
  const uint32_t xo = ss_off<T>(vx, st, sc), dto = ss_off<T>(a.dt, st, sc), zo = ss_off<T>(a.z, st, sc), Bo = ss_off<T>(vb, bt, bn);
  float bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) bias[v] = a.bias && sok ? a.bias[u.c0 + sc + v] : 0.0f;
  SsRaw<T, V> xn = {}, dn = {}, zn = {};
  SsRaw<T, VB> Bn = {};
  const int tiles = (s.len + TT - 1) / TT;
  const int t1 = s.t0 + (REV && tiles ? (tiles - 1) * TT : 0), way = REV ? -TT : TT;
  const char *xp = ss_tile_at<T>(vx, s.vb, t1, u.c0), *dp = ss_tile_at<T>(a.dt, s.vb, t1, u.c0), *zp = ss_tile_at<T>(a.z, s.vb, t1, u.c0);
  const char* Bp = ss_tile_at<T>(vb, s.vb, t1, u.g * vb.sh);
  auto fetch = [&](int t) {
    if (sok && t + st < s.len) {
      ss_load_at(xn, xp, xo);
      ss_load_at(dn, dp, dto);
      if (gated) ss_load_at(zn, zp, zo);
    }
    if (bok && t + bt < s.len) ss_load_at(Bn, Bp, Bo);
    xp += ss_rows<T>(vx, way);
    dp += ss_rows<T>(a.dt, way);
    zp += ss_rows<T>(a.z, way);
    Bp += ss_rows<T>(vb, way);
  };
  auto at = [&](int i) { return (REV ? tiles - 1 - i : i) * TT; };
  if (tiles) fetch(at(0));
  double total = 0.0;   // (long sums of steps: fp32 inside a tile)
  const int wblk = u.c0 % (a.D / a.G) / CW + wave;   // wave's channel block in its group
  const int nblk = (a.D / a.G + CW - 1) / CW;
  for (int i = 0; i < tiles; ++i) {
    const int t0 = at(i), p = i & 1;
    const bool live = sok && t0 + st < s.len, blive = bok && t0 + bt < s.len;
    float d[V], x[V], none[V];
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = dn.get(v) + bias[v];
    ss_steps<V, false>(d, none, a.softplus, live);
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = REV ? (live ? xn.get(v) : 0.0f) : d[v] * xn.get(v);
    if (gated) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float z = zn.get(v);
        x[v] *= z * ss_sigmoid<T>(z);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) du[p][st][sc + v] = make_float2(d[v], x[v]);
    if (tid < BT) {
      SsVec<float, VB> b;
#pragma unroll
      for (int v = 0; v < VB; ++v) b.e[v] = blive ? Bn.get(v) : 0.0f;
      *(SsVec<float, VB>*)&Bs[p][bt][bn] = b;
    }
    __syncthreads();
    if (i + 1 < tiles) fetch(at(i + 1));
    if (!REV && a.ckpt && t0 % kSsBwdTile == 0) {
      const int64_t tile = ss_tile(a, s.b, u.sid, s.t0, t0);
      if (wblk < nblk) ss_lane_put(a.ckpt + ((tile * a.G + u.g) * nblk + wblk) * (S * 64), h, lane);
      if (ok && q == 0) a.cum[tile * a.D + ch] = ss_held_sum((float)total);
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
  if (!REV && ok && q == 0) a.sum[(int64_t)u.sid * a.D + ch] = ss_held_sum((float)total);
}

// Both directions in one launch (z), as neither waits for the other.
template <typename T, int S, int NS>
__global__ __launch_bounds__(256) void pdssm_selscan_state_kernel(const SsArgs a) {
  __shared__ SsStateLds<S, NS> lds;
  if (blockIdx.z)
    ss_state_body<T, S, NS, true>(a, lds);
  else
    ss_state_body<T, S, NS, false>(a, lds);
}

// ---- gradient
//
//   l_t = g_t C_t + a_{t+1} l_{t+1}                    g = g_y silu(z)
//   g_C = sum_d g h        g_B = sum_d l (d x)         g_x = g D + d (l . B)
//   g_d = x (l . B) + sum_n A q h_{t-1}                q = a_t l_t
//   g_A = sum_t d q h_{t-1}
//
// Tiles of 32 steps from the run's end, each from the state at its start
// (the state pass wrote it, from its piece's start): four waves take eight
// steps each, forwards and backwards from zero first, then, with what enters
// at both ends, again on the decays and states in registers.
//
// Sums over the channels (g_B, g_C) are the part that crosses lanes: for every
// step and state, over the 16 lanes that hold channels.  Exchanges halve what is
// left of four steps' products twice, so that only a quarter of them is added
// up inside the rows of 16 lanes.  (On the matrix cores, as products with a row
// of ones, they took 32 cycles each: 660 us for the kernel below.)
//
// 16 x 2048 x 768 x 16 in bf16: the whole gradient 529 us; this kernel 460 to 505 under
// the profiler, 387 of them the vector units: 61000 instructions a wave for its 64 tiles of 32 cells a
// lane, three waves a SIMD.  The tile's outputs leave before the next is
// staged: with two tiles' rows in LDS and two barriers the gradient took 690 us instead of 590.
//
// No register of it may be spilled.  A reload in the loop waits for every load
// under way (592 us, and 191 instead of 164 for 9 packed in 4097 x 512 x 32), and a
// value stored to scratch where only some lanes are on can come back as something else in
// the others: addresses, here.  So offsets and, where there is no room, indexes
// are formed where they are used.
template <typename T, int S, int NS>
__global__ __launch_bounds__(256, S >= 8 ? 2 : 3) void pdssm_selscan_bwd_kernel(const SsArgs a) {
  constexpr int W = kSsTimeWaves, TS = kSsBwdSteps, TT = W * TS, CC = 64 / NS, NP = S * NS;
  constexpr int V = TT * CC / 256;
  constexpr int BT = 128, VB = TT * NP / BT < 8 ? TT * NP / BT : 8, BR = TT * NP / BT / VB;   // B by one half of the threads, C by the other
  static_assert(kSsBwdGroups == 1 && TS % 4 == 0, "a workgroup's waves share their channels; sums over them take four steps at once");
  __shared__ __align__(16) float4 pre[TT][CC];     // d, d x, g, slope of d
  __shared__ __align__(16) float gzs[TT][CC];      // slope of the gate times g_y
  __shared__ __align__(16) float Bs[TT][NP], Cs[TT][NP];
  __shared__ float outs[3 * (TT * CC + 16)];       // C . h, l . B, sum A q h: 16 banks apart
  __shared__ __align__(16) float gs[2][TT][NP];   // g_B, g_C
  __shared__ __align__(16) float Es[W][S * 64], Ps[W][S * 64], Rs[W][S * 64];
  __shared__ __align__(16) float Rt[2][S * 64];   // the adjoint state that enters a tile, from its end
  constexpr bool kPark = S >= 8;   // 256 registers do not hold everything: the entering states of a wave's steps lie here meanwhile
  __shared__ __align__(16) float Hin[kPark ? W : 1][kPark ? S * 64 : 4];
  __shared__ __align__(16) float pars[2][CC];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6) % W;   // (so that the compiler knows its range: 531 -> 529 us)
  if (ss_block(a.row) == 0 && tid < 2) a.header[tid] = 0;
  SsUnit u;
  if (!ss_unit(a, CC, u)) return;
  SsSeg s;
  const int lc = lane / NS, q = lane % NS, ch = u.c0 + lc;
  const bool ok = ch < u.end;
  const bool found = ss_segment(a.s, u.sid, s);
  float* partA = a.partA + (int64_t)u.sid * a.D * (a.N + 2);
  if (!found || s.len <= 0) {   // no rows: nothing but sums of none and what passes through
    const float zero[S] = {};
    if (wave == 0) {
      ss_store_state(zero, partA, ch, q * S, a.N, ok);
      if (ok && q < 2) partA[(int64_t)a.D * (a.N + q) + ch] = 0.0f;
      if (found && s.first && a.gh0) {
        float r[S];
        ss_load_state(r, a.ghL, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
        ss_store_state(r, a.gh0, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
      }
    }
    return;
  }
  const int piece0 = ss_piece(a, s, u.sid);
  float A2[S], gA[S];
  ss_load_A(A2, a.A, ch, q * S, a.N, ok);
  if (wave == 0) {
    float R[S];
    if (s.last)
      ss_load_state(R, a.ghL, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
    else
      ss_load_state(R, a.adj, (int64_t)ss_piece_at(piece0, (s.len - 1) / a.piece, a.npieces) * a.D + ch, q * S, a.N, ok);
    ss_lane_put(Rt[0], R, lane);
  }
#pragma unroll
  for (int j = 0; j < S; ++j) gA[j] = 0.0f;

  // Where a thread stages and stores: a step's V channels; VB states of B or C, and rows BT VB / NP further on.
  // With eight states a lane there is no room to hold it through the loop.
  struct At { int st, sc, bt, bn; };
  auto where = [](int i) { return At{i * V / CC, i * V % CC, i % BT * VB / NP, i % BT * VB % NP}; };
  const At held = where(tid);
  auto here = [&] { return S < 8 ? held : where(ss_thread_here()); };
  const bool second = __builtin_amdgcn_readfirstlane(tid >> 6) >= BT / 64, sok = u.c0 + here().sc < u.end, gated = a.z.p != nullptr;
  const bool bok = here().bn < a.N;
  // (whole waves take B or C; by value: a reference would be followed through memory in every tile)
  LaView vbc;
  vbc.p = second ? a.Cm.p : a.Bm.p;
  vbc.sb = second ? a.Cm.sb : a.Bm.sb;
  vbc.sh = second ? a.Cm.sh : a.Bm.sh;
  vbc.st = second ? a.Cm.st : a.Bm.st;
  constexpr int BS = BT * VB / NP;
  if (tid < CC) {
    const int k = u.c0 + tid;
    pars[0][tid] = a.bias && k < u.end ? a.bias[k] : 0.0f;
    pars[1][tid] = a.skip && k < u.end ? a.skip[k] : 0.0f;
  }
  __syncthreads();
  float gD[V], gb[V];
#pragma unroll
  for (int v = 0; v < V; ++v) gD[v] = gb[v] = 0.0f;
  const int wblk = u.c0 % (a.D / a.G) / CC, nblk = (a.D / a.G + CC - 1) / CC;
  SsRaw<T, V> xn = {}, dn = {}, zn = {}, gn = {};
  SsRaw<T, VB> Bn[BR] = {};
  const int last = (s.len - 1) / TT * TT, t1 = s.t0 + last;
  const char *xp = ss_tile_at<T>(a.x, s.vb, t1, u.c0), *dp = ss_tile_at<T>(a.dt, s.vb, t1, u.c0), *zp = ss_tile_at<T>(a.z, s.vb, t1, u.c0);
  const char *gp = ss_tile_at<T>(a.gy, s.vb, t1, u.c0), *Bp = ss_tile_at<T>(vbc, s.vb, t1, u.g * vbc.sh);
  char *gxp = ss_tile_at<T>(a.gx, s.vb, t1, u.c0), *gdp = ss_tile_at<T>(a.gdt, s.vb, t1, u.c0), *gzp = ss_tile_at<T>(a.gz, s.vb, t1, u.c0);
  auto fetch = [&](int t) {   // and the pointers back to the tile before it
    const auto [st, sc, bt, bn] = here();
    if (sok && t + st < s.len) {
      ss_load_at(xn, xp, ss_off_here<T>(a.x, st, sc));
      ss_load_at(dn, dp, ss_off_here<T>(a.dt, st, sc));
      ss_load_at(gn, gp, ss_off_here<T>(a.gy, st, sc));
      if (gated) ss_load_at(zn, zp, ss_off_here<T>(a.z, st, sc));
    }
#pragma unroll
    for (int i = 0; i < BR; ++i)
      if (bok && t + bt + i * BS < s.len) ss_load_at(Bn[i], Bp + ss_rows<T>(vbc, i * BS), ss_off_here<T>(vbc, bt, bn));
    xp -= ss_rows<T>(a.x, TT);
    dp -= ss_rows<T>(a.dt, TT);
    gp -= ss_rows<T>(a.gy, TT);
    zp -= ss_rows<T>(a.z, TT);
    Bp -= ss_rows<T>(vbc, TT);
  };
  int pc = __builtin_amdgcn_readfirstlane((s.len - 1) / a.piece), turn = 0;   // piece of the tile
  auto arrived = [&] {
    ss_arrived(xn);
    ss_arrived(dn);
    ss_arrived(zn);
    ss_arrived(gn);
#pragma unroll
    for (int i = 0; i < BR; ++i) ss_arrived(Bn[i]);
  };
  fetch(last);
  arrived();
  for (int t0 = last; t0 >= 0; t0 -= TT, turn ^= 1) {
    const auto [st, sc, bt, bn] = here();
    const bool live = sok && t0 + st < s.len;
    const SsRaw<T, V> xc = xn;
    float d[V], sg[V], g[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      d[v] = dn.get(v) + pars[0][sc + v];
      g[v] = gn.get(v);   // (behind the end, which the first tile has, nothing was loaded: zero)
    }
    ss_steps<V, true>(d, sg, a.softplus, live);
    if (gated) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float z = zn.get(v), k = ss_sigmoid<T>(z);
        gzs[st][sc + v] = g[v] * k * __builtin_fmaf(z, 1.0f - k, 1.0f);
        g[v] *= z * k;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) pre[st][sc + v] = make_float4(d[v], d[v] * xc.get(v), g[v], sg[v]);
#pragma unroll
    for (int i = 0; i < BR; ++i) {
      const int t = bt + i * BS;
      SsVec<float, VB> b;
#pragma unroll
      for (int v = 0; v < VB; ++v) b.e[v] = Bn[i].get(v);
      *(SsVec<float, VB>*)(second ? &Cs[t][bn] : &Bs[t][bn]) = b;
    }
    __syncthreads();
    if (t0) fetch(t0 - TT);
    // the state at the tile's start: what it was from its piece's start, and what entered there
    if (t0 < pc * a.piece) --pc;
    const int at = ss_piece_at(piece0, pc, a.npieces);
    const int64_t tile = ss_tile(a, s.b, at, s.t0 + pc * a.piece, t0 - pc * a.piece);
    float hin[S] = {}, H0[S], cum = 0.0f;
    {
      const int ln = S < 8 && sizeof(typename T::E) == 2 ? lane : ss_thread_here() & 63, k = ln / NS;
      const bool has = u.c0 + k < u.end;
      if (wblk < nblk) ss_lane_get(hin, a.ckpt + ((tile * a.G + u.g) * nblk + wblk) * (S * 64), ln);
      if (has) cum = (a.cum + tile * a.D + u.c0)[k];
      const float* entered = a.seg ? a.seg + ((int64_t)at * a.D + u.c0) * a.N : a.h0 ? a.h0 + ((int64_t)s.b * a.D + u.c0) * a.N : nullptr;
      ss_load_state(H0, entered, k, ln % NS * S, a.N, has);
    }

    // from zero, forwards and backwards
    const int tw = wave * TS;
    float dec[TS][S], hs[TS][S], h[S], l[S], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < S; ++j) h[j] = l[j] = 0.0f;
#pragma unroll
    for (int t4 = 0; t4 < TS; t4 += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t4 + i;
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
      __builtin_amdgcn_sched_barrier(0);
    }
    ss_lane_put(Es[wave], h, lane);
    sum = ss_held_sum(sum);
#pragma unroll
    for (int j = 0; j < S; ++j) h[j] = ss_exp2(sum * A2[j]);
    ss_lane_put(Ps[wave], h, lane);
#pragma unroll
    for (int t4 = TS - 4; t4 >= 0; t4 -= 4) {
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const int t = t4 + i;
        const float g1 = pre[tw + t][lc].z;
        float k[S];
        ss_row_get(k, &Cs[tw + t][q * S]);
#pragma unroll
        for (int j = 0; j < S; ++j) l[j] = dec[t][j] * __builtin_fmaf(g1, k[j], l[j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    ss_lane_put(Rs[wave], l, lane);
    __syncthreads();
    // what enters at both ends of this wave's steps; the first wave's adjoint leaves the tile then
#pragma unroll
    for (int j = 0; j < S; ++j) hin[j] = __builtin_fmaf(ss_exp2(cum * A2[j]), H0[j], hin[j]);
#pragma unroll
    for (int v = 0; v < W - 1; ++v) {
      if (v < wave) {
        float e[S], p[S];
        ss_lane_get(e, Es[v], lane);
        ss_lane_get(p, Ps[v], lane);
#pragma unroll
        for (int j = 0; j < S; ++j) hin[j] = __builtin_fmaf(p[j], hin[j], e[j]);
      }
    }
    {
      float r[S], p[S];   // own contribution and decay, for the first wave
#pragma unroll
      for (int j = 0; j < S; ++j) {
        r[j] = l[j];
        p[j] = h[j];
      }
      ss_lane_get(l, Rt[turn], lane);
#pragma unroll
      for (int v = W - 1; v > 0; --v) {
        if (v > wave) {
          float e[S], f[S];
          ss_lane_get(e, Rs[v], lane);
          ss_lane_get(f, Ps[v], lane);
#pragma unroll
          for (int j = 0; j < S; ++j) l[j] = __builtin_fmaf(f[j], l[j], e[j]);
        }
      }
      if (wave == 0) {
#pragma unroll
        for (int j = 0; j < S; ++j) r[j] = __builtin_fmaf(p[j], l[j], r[j]);
        ss_lane_put(Rt[turn ^ 1], r, lane);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < S; ++j) h[j] = hin[j];
#pragma unroll
    for (int t = 0; t < TS; ++t)
#pragma unroll
      for (int j = 0; j < S; ++j) hs[t][j] = h[j] = __builtin_fmaf(dec[t][j], h[j], hs[t][j]);
    if constexpr (kPark) ss_lane_put(Hin[wave], hin, lane);
    float far[2][2 * S];   // products of the two steps before: g_B's S, then g_C's
#pragma unroll
    for (int t = TS - 1; t >= 0; --t) {
      const float4 w = pre[tw + t][lc];
      float b[S], k[S], y = 0.0f, lb = 0.0f, pa = 0.0f, v[2 * S];
      if constexpr (kPark)
        if (t == 0) ss_lane_get(hin, Hin[wave], lane);
      ss_row_get(b, &Bs[tw + t][q * S]);
      ss_row_get(k, &Cs[tw + t][q * S]);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        l[j] = __builtin_fmaf(w.z, k[j], l[j]);
        v[j] = w.y * l[j];
        v[S + j] = w.z * hs[t][j];
        y = __builtin_fmaf(k[j], hs[t][j], y);
        lb = __builtin_fmaf(b[j], l[j], lb);
        l[j] *= dec[t][j];
        const float p = l[j] * (t ? hs[t ? t - 1 : 0][j] : hin[j]);
        pa = __builtin_fmaf(A2[j], p, pa);
        gA[j] = __builtin_fmaf(w.x, p, gA[j]);
      }
      // over the states, lanes next to each other: the sum of y ends in lane 0 of four, of lb in 1, of pa in 2
      const bool odd = q & 1, high = q & 2;
      const float r1 = (odd ? lb : y) + ss_dpp<kDppXor1>(odd ? y : lb);
      const float r2 = pa + ss_dpp<kDppXor1>(pa);
      float r = (high ? r2 : r1) + ss_dpp<kDppXor2>(high ? r1 : r2);
      if constexpr (NS == 8) r += ss_dpp<kDppShl4>(r);
      if (q < 3) outs[q * (TT * CC + 16) + (tw + t) * CC + lc] = r;
      // over the channels: lanes 32 apart, rows, then what is left of a row; four steps end in a row each
      if (t % 4 >= 2) {
#pragma unroll
        for (int j = 0; j < 2 * S; ++j) far[t & 1][j] = v[j];
      } else {
        ss_fold32(far[t & 1], v, far[t & 1]);
      }
      if (t % 4 == 0) {
        float g[2 * S];
        ss_fold16(g, far[0], far[1]);
        const int at = tw + t + (lane >> 4);
#pragma unroll
        for (int j = 0; j < 2 * S; ++j) {
          g[j] += ss_dpp<kDppRor8>(g[j]);
          if constexpr (NS == 4) g[j] += ss_dpp<kDppRor4>(g[j]);
        }
        if ((lane & 15) < NS) {
          constexpr int U = S < 4 ? S : 4;
#pragma unroll
          for (int j = 0; j < 2 * S; j += U) {
            SsVec<float, U> o;
#pragma unroll
            for (int i = 0; i < U; ++i) o.e[i] = g[j + i];
            *(SsVec<float, U>*)&gs[j / S][at][q * S + j % S] = o;
          }
        }
      }
      if (t % 2 == 0) __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    // The next tile's rows are here by now.  Waited for before anything is
    // stored: behind the stores, the wait would be for them too.
    arrived();
    {
      const auto [st, sc, bt, bn] = here();
      if (live) {
        float ox[V], od[V], oz[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float4 w = pre[st][sc + v];
          const float* o = outs + st * CC + sc + v;
          const float y = o[0], lb = o[TT * CC + 16], pa = kLn2 * o[2 * (TT * CC + 16)];
          const float x = xc.get(v), skip = pars[1][sc + v];
          ox[v] = __builtin_fmaf(w.x, lb, w.z * skip);
          od[v] = __builtin_fmaf(x, lb, pa) * w.w;
          oz[v] = gated ? gzs[st][sc + v] * __builtin_fmaf(skip, x, y) : 0.0f;
          gD[v] = __builtin_fmaf(w.z, x, gD[v]);
          gb[v] += od[v];
        }
        ss_store_at<T, V>(gxp, ss_off_here<T>(a.gx, st, sc), ox);
        ss_store_at<T, V>(gdp, ss_off_here<T>(a.gdt, st, sc), od);
        if (gated) ss_store_at<T, V>(gzp, ss_off_here<T>(a.gz, st, sc), oz);
      }
      gxp -= ss_rows<T>(a.gx, TT);
      gdp -= ss_rows<T>(a.gdt, TT);
      gzp -= ss_rows<T>(a.gz, TT);
      // this workgroup's part of g_B (first half of the threads) and g_C
#pragma unroll
      for (int i = 0; i < BR; ++i) {
        const int t = bt + i * BS;
        if (!bok || t0 + t >= s.len) continue;
        const int nb = a.G * ((a.D / a.G + CC - 1) / CC);
        const int64_t r = s.vb * a.s.L + s.t0 + t0 + t;
        float* o = a.part + ((((int64_t)(second ? nb : 0) + u.block) * a.rows) + r) * a.N + bn;
        SsVec<float, VB> v;
#pragma unroll
        for (int j = 0; j < VB; ++j) v.e[j] = gs[second][t][bn + j];
        *(SsVec<float, VB>*)o = v;
      }
    }
  }
  {   // (nothing of this is held through the loop)
    const int i = ss_thread_here(), lane = i & 63, lc = lane / NS, q = lane % NS, ch = u.c0 + lc;
    const bool ok = ch < u.end;
    const auto [st, sc, bt, bn] = where(i);
    if (s.first && wave == 0 && a.gh0) {
      float R[S];
      ss_lane_get(R, Rt[turn], lane);
      ss_store_state(R, a.gh0, (int64_t)s.b * a.D + ch, q * S, a.N, ok);
    }
    // sums over this workgroup's steps: the four waves', then the staging threads' of every channel
    __syncthreads();
    ss_lane_put(Es[wave], gA, lane);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      outs[st * CC + sc + v] = gD[v];
      outs[TT * CC + 16 + st * CC + sc + v] = gb[v];
    }
    __syncthreads();
    if (wave == 0) {
      float sumA[S], e[S];
      ss_lane_get(sumA, Es[0], lane);
      for (int v = 1; v < W; ++v) {
        ss_lane_get(e, Es[v], lane);
#pragma unroll
        for (int j = 0; j < S; ++j) sumA[j] += e[j];
      }
      ss_store_state(sumA, partA, ch, q * S, a.N, ok);
      if (ok && q < 2) {
        float o = 0.0f;
        for (int t = 0; t < TT; ++t) o += outs[q * (TT * CC + 16) + t * CC + lc];
        partA[(int64_t)a.D * (a.N + q) + ch] = o;
      }
    }
  }
}

// ---- one token
//
// Four states a lane, a channel in neighbouring lanes: the state streams
// through in whole lines, once each way, which is the time (250 rows of 2048 x
// 16: 69 MB in 17 us).  Everything is under way before the search for an
// earlier row of the same slot.
template <typename T, int NS>
__global__ __launch_bounds__(256) void pdssm_selscan_step_kernel(const SsStepArgs a) {
  constexpr int CW = 256 / NS;
  const int tid = threadIdx.x, nb = (a.D + CW - 1) / CW;
  const unsigned id = ss_block(a.row);
  const int b = id / nb, ch = id % nb * CW + tid / NS, q = tid % NS, n0 = q * 4;
  if (b >= a.B) return;
  const int slot = a.idx ? a.idx[b] : b;
  const bool ok = ch < a.D, has = ok && n0 < a.N && slot >= 0 && slot < a.slots;
  float* hp = a.state + ((int64_t)slot * a.D + ch) * a.N + n0;
  float4 h = make_float4(0, 0, 0, 0), A = h;
  SsRaw<T, 4> vb = {}, vc = {};
  float x = 0.0f, raw = 0.0f, z = 0.0f, skip = 0.0f;
  if (has) {
    h = *(const float4*)hp;
    const int g = ch / (a.D / a.G);
    A = *(const float4*)(a.A + (int64_t)ch * a.N + n0);
    ss_load_raw(vb, a.Bm.p, (int64_t)b * a.Bm.sb + (int64_t)g * a.Bm.sh + n0);
    ss_load_raw(vc, a.Cm.p, (int64_t)b * a.Cm.sb + (int64_t)g * a.Cm.sh + n0);
    x = T::get(((const typename T::E*)a.x.p)[(int64_t)b * a.x.sb + ch]);
    raw = T::get(((const typename T::E*)a.dt.p)[(int64_t)b * a.dt.sb + ch]) + (a.bias ? a.bias[ch] : 0.0f);
    if (a.z.p) z = T::get(((const typename T::E*)a.z.p)[(int64_t)b * a.z.sb + ch]);
    skip = a.skip ? a.skip[ch] : 0.0f;
  }
  if (ss_taken(a.idx, b, slot, a.slots, tid & 63)) {
    const float f = slot < 0 ? 0.0f : __builtin_nanf("");
    if (ok && q == 0) ss_store<T, 1>(a.y.p, (int64_t)b * a.y.sb + ch, &f);
    return;
  }
  const float d = a.softplus ? ss_softplus_of(raw, ss_decay(raw)) : raw, u = d * x, w = ss_held_sum(d * kLog2e);
  h.x = __builtin_fmaf(ss_exp2(w * A.x), h.x, u * vb.get(0));
  h.y = __builtin_fmaf(ss_exp2(w * A.y), h.y, u * vb.get(1));
  h.z = __builtin_fmaf(ss_exp2(w * A.z), h.z, u * vb.get(2));
  h.w = __builtin_fmaf(ss_exp2(w * A.w), h.w, u * vb.get(3));
  if (has) *(float4*)hp = h;
  float y = has ? (vc.get(0) * h.x + vc.get(1) * h.y) + (vc.get(2) * h.z + vc.get(3) * h.w) : 0.0f;
  y += ss_dpp<kDppXor1>(y);
  if constexpr (NS >= 4) y += ss_dpp<kDppXor2>(y);
  if constexpr (NS >= 8) y += ss_dpp<kDppHalfMirror>(y);
  if constexpr (NS >= 16) y += ss_dpp<kDppRor8>(y);
  if (ok && q == 0) {
    y = __builtin_fmaf(skip, x, y);
    if (a.z.p) y *= z * ss_sigmoid<T>(z);
    ss_store<T, 1>(a.y.p, (int64_t)b * a.y.sb + ch, &y);
  }
}

}  // namespace pdscan
