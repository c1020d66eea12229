// Launchers of the selective scan, and its small kernels: the carry between
// segments and the sums that finish a gradient.
#include <type_traits>

#include "pdscan_selscan.h"
#include "pdscan_ssm_launch.h"

namespace pdscan {

// Entering states of all pieces of a sequence from the pieces' contributions,
// in place: four states of a channel a thread, eight pieces' loads at once; backwards (z) the adjoint's.
__global__ __launch_bounds__(256) void pdssm_selscan_carry_kernel(const SsCarryArgs a) {
  const unsigned id = ss_block(a.row);
  const int b = id / a.blocks, rev = blockIdx.z;
  const int64_t e = ((int64_t)(id % a.blocks) * 256 + threadIdx.x) * 4, state = (int64_t)a.D * a.N;
  if (b >= a.B || e >= state) return;
  const int ch = (int)(e / a.N);
  const int s0 = a.starts ? a.starts[b] : b * a.npiece, s1 = a.starts ? a.starts[b + 1] : s0 + a.npiece, n = s1 - s0;
  float4 A = *(const float4*)(a.A + e), S = make_float4(0, 0, 0, 0);
  A = make_float4(ss_held_decay(A.x * kLog2e), ss_held_decay(A.y * kLog2e), ss_held_decay(A.z * kLog2e), ss_held_decay(A.w * kLog2e));
  float* seg = a.seg[rev];
  if (a.user[rev]) S = *(const float4*)(a.user[rev] + b * state + e);
  constexpr int U = 8;
  for (int i0 = 0; i0 < n; i0 += U) {
    float4 v[U];
    float d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u < n ? i0 + u : n - 1;
      const int64_t at = rev ? s1 - 1 - i : s0 + i;
      v[u] = *(const float4*)(seg + at * state + e);
      d[u] = a.sum[at * a.D + ch];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= n) break;
      const int64_t at = rev ? s1 - 1 - (i0 + u) : s0 + i0 + u;
      *(float4*)(seg + at * state + e) = S;
      S.x = __builtin_fmaf(ss_exp2(d[u] * A.x), S.x, v[u].x);
      S.y = __builtin_fmaf(ss_exp2(d[u] * A.y), S.y, v[u].y);
      S.z = __builtin_fmaf(ss_exp2(d[u] * A.z), S.z, v[u].z);
      S.w = __builtin_fmaf(ss_exp2(d[u] * A.w), S.w, v[u].w);
    }
  }
}

// Sums over parts p0 .. p1 - 1, in one order: 64 columns a workgroup, every fourth part a wave.
__device__ __forceinline__ void ss_sum_columns(const SsSumArgs& a, int64_t block, int p0, int p1, float* to) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t i = block * 64 + lane;
  float x = 0.0f;
  if (i < a.width) {
#pragma unroll 8
    for (int p = p0 + wave; p < p1; p += 4) x += a.part[(int64_t)p * a.width + i];
  }
  red[wave][lane] = x;
  __syncthreads();
  if (wave || i >= a.width) return;
  x = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
  if (to) {
    to[i] = x;
    return;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (i < a.share[k]) {
      if (a.out[k]) a.out[k][i] = x;
      return;
    }
    i -= a.share[k];
  }
}

// Where there are many parts, kSsSumMid runs of them first (y).
__global__ __launch_bounds__(256) void pdssm_ssm_sum_kernel(const SsSumArgs a, int each, float* mid) {
  const int p0 = blockIdx.y * each, p1 = a.parts - p0 < each ? a.parts : p0 + each;
  ss_sum_columns(a, blockIdx.x, p0, p1, mid ? mid + blockIdx.y * a.width : nullptr);
}

// g_B (first workgroups) and g_C from the channel blocks' parts, each read
// once (33 us for 201 MB), and behind them the sums over the runs.
template <typename T>
__global__ __launch_bounds__(256) void pdssm_selscan_fold_kernel(const SsFoldArgs a) {
  if (blockIdx.x >= 2 * a.folds) {
    ss_sum_columns(a.sum, blockIdx.x - 2 * a.folds, 0, a.sum.parts, nullptr);
    return;
  }
  const int n4 = a.N / 4, y = blockIdx.x >= a.folds;
  const unsigned block = blockIdx.x - y * a.folds;
  int64_t r0 = 0, r1 = a.rows;
  if (a.cu) {   // rows outside the sequences stay as they are
    r0 = a.cu[0];
    r1 = a.cu[a.B];
    r0 = r0 < 0 ? 0 : r0 > a.rows ? a.rows : r0;
    r1 = r1 < r0 ? r0 : r1 > a.rows ? a.rows : r1;
  }
  const int64_t n = (r1 - r0) * a.G * n4, step = (int64_t)a.rows * a.N;
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < n; i += (int64_t)a.folds * 256) {
    // rows next to each other along a block's part
    const int c = (int)(i % n4) * 4;
    const int64_t row = r0 + i / n4 % (r1 - r0);
    const int g = (int)(i / n4 / (r1 - r0));
    const float* p = a.part + ((int64_t)y * a.G * a.blocks + (int64_t)g * a.blocks) * step + row * a.N + c;
    float v[4] = {0, 0, 0, 0};
#pragma unroll 8
    for (int k = 0; k < a.blocks; ++k) {
      const float4 w = *(const float4*)(p + k * step);
      v[0] += w.x; v[1] += w.y; v[2] += w.z; v[3] += w.w;
    }
    const LaView& o = a.out[y];
    const int64_t b = a.cu ? 0 : row / a.L, t = a.cu ? row : row % a.L;
    ss_store<T, 4>(o.p, b * o.sb + g * o.sh + t * o.st + c, v);
  }
}

namespace {

template <typename F>
hipError_t by_states(int N, F f) {   // f(S, NS) as constants
  if (N <= 8) f(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
  else if (N <= 16) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
  else if (N <= 32) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
  return hipGetLastError();
}

LaGrid units(SsArgs& a, int per, int threads) {
  const long long n = (long long)a.s.segs * a.G * ss_blocks(a.D / a.G, per);
  const LaGrid g = la_grid_rows((n + 7) / 8 * 8, threads);
  a.row = g.x;
  return g;
}

}  // namespace

hipError_t launch_selscan_fwd(const SsArgs& args, int bf16, hipStream_t st) {
  SsArgs a = args;
  const LaGrid g = units(a, ss_channels(a.N), 256);
  return by_states(a.N, [&](auto s, auto ns) {
    constexpr int S = decltype(s)::value, NS = decltype(ns)::value, TS = kSsFwdSteps;
    if (bf16)
      hipLaunchKernelGGL((pdssm_selscan_kernel<SsBf16, S, NS, TS>), dim3(g.x, g.y), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((pdssm_selscan_kernel<SsF32, S, NS, TS>), dim3(g.x, g.y), dim3(256), 0, st, a);
  });
}

hipError_t launch_selscan_state(const SsArgs& args, int bf16, hipStream_t st) {
  SsArgs a = args;
  const LaGrid g = units(a, ss_channels(a.N) * kSsStateGroups, 256);
  const unsigned both = a.adj ? 2 : 1;
  return by_states(a.N, [&](auto s, auto ns) {
    constexpr int S = decltype(s)::value, NS = decltype(ns)::value;
    if (bf16)
      hipLaunchKernelGGL((pdssm_selscan_state_kernel<SsBf16, S, NS>), dim3(g.x, g.y, both), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((pdssm_selscan_state_kernel<SsF32, S, NS>), dim3(g.x, g.y, both), dim3(256), 0, st, a);
  });
}

hipError_t launch_selscan_bwd(const SsArgs& args, int bf16, hipStream_t st) {
  SsArgs a = args;
  const LaGrid g = units(a, ss_channels(a.N), 256);
  return by_states(a.N, [&](auto s, auto ns) {
    constexpr int S = decltype(s)::value, NS = decltype(ns)::value;
    if (bf16)
      hipLaunchKernelGGL((pdssm_selscan_bwd_kernel<SsBf16, S, NS>), dim3(g.x, g.y), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((pdssm_selscan_bwd_kernel<SsF32, S, NS>), dim3(g.x, g.y), dim3(256), 0, st, a);
  });
}

hipError_t launch_selscan_carry(const SsCarryArgs& args, hipStream_t st) {
  SsCarryArgs a = args;
  a.blocks = (int)(((long long)a.D * a.N + 1023) / 1024);
  const LaGrid g = la_grid_rows((long long)a.B * a.blocks, 256);
  a.row = g.x;
  hipLaunchKernelGGL(pdssm_selscan_carry_kernel, dim3(g.x, g.y, a.seg[1] ? 2 : 1), dim3(256), 0, st, a);
  return hipGetLastError();
}

namespace {

// Leaves at most kSsSumMost parts.
void sum_many(SsSumArgs& a, hipStream_t st) {
  if (a.parts <= kSsSumMost) return;
  const int each = (a.parts + kSsSumMid - 1) / kSsSumMid;
  hipLaunchKernelGGL(pdssm_ssm_sum_kernel, dim3((unsigned)((a.width + 63) / 64), kSsSumMid), dim3(256), 0, st, a, each, a.mid);
  a.part = a.mid;
  a.parts = kSsSumMid;
}

}  // namespace

hipError_t launch_selscan_fold(const SsFoldArgs& args, int bf16, hipStream_t st) {
  SsFoldArgs a = args;
  sum_many(a.sum, st);
  const long long folds = (a.rows * a.G * (a.N / 4) + 255) / 256;
  a.folds = folds > 4096 ? 4096 : (unsigned)folds;
  const unsigned grid = 2 * a.folds + (unsigned)((a.sum.width + 63) / 64);
  if (bf16)
    hipLaunchKernelGGL(pdssm_selscan_fold_kernel<SsBf16>, dim3(grid), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(pdssm_selscan_fold_kernel<SsF32>, dim3(grid), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_ssm_sum(const SsSumArgs& args, hipStream_t st) {
  SsSumArgs a = args;
  sum_many(a, st);
  hipLaunchKernelGGL(pdssm_ssm_sum_kernel, dim3((unsigned)((a.width + 63) / 64)), dim3(256), 0, st, a, a.parts, (float*)nullptr);
  return hipGetLastError();
}

hipError_t launch_selscan_step(const SsStepArgs& args, int bf16, hipStream_t st) {
  SsStepArgs a = args;
  const int ns = a.N <= 8 ? 2 : a.N <= 16 ? 4 : a.N <= 32 ? 8 : 16, cw = 256 / ns;
  const LaGrid g = la_grid_rows((long long)a.B * ((a.D + cw - 1) / cw), 256);
  a.row = g.x;
  auto go = [&](auto n) {
    constexpr int NS = decltype(n)::value;
    if (bf16)
      hipLaunchKernelGGL((pdssm_selscan_step_kernel<SsBf16, NS>), dim3(g.x, g.y), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((pdssm_selscan_step_kernel<SsF32, NS>), dim3(g.x, g.y), dim3(256), 0, st, a);
  };
  if (ns == 2) go(std::integral_constant<int, 2>{});
  else if (ns == 4) go(std::integral_constant<int, 4>{});
  else if (ns == 8) go(std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 16>{});
  return hipGetLastError();
}

}  // namespace pdscan
