// Segment table of packed sequences.  Included behind what defines the kernel
// language: <hip/hip_runtime.h>, or a test's stand-ins on the host.
#pragma once

#include <cstdint>

namespace pdscan {

// Segments of packed sequences, in order: {sequence, first row, rows,
// first | last << 1}, then the first segment of every sequence.  Every
// sequence has at least one segment (an empty one passes its state through);
// entries behind the last hold -1 rows.  One workgroup, 3 to 5 us: its launch.
__global__ __launch_bounds__(256) void pdssm_linattn_table_kernel(const int32_t* cu, int32_t* table,
                                                                  int32_t* starts, int B, int L, int seg, int segs) {
  __shared__ long long wsum[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  long long base = 0;   // offsets out of order can ask for more segments than 32 bits count
  for (int b0 = 0; b0 < B; b0 += 256) {
    const int b = b0 + tid;
    int t0 = 0, len = 0, n = 0;
    if (b < B) {
      t0 = cu[b];
      int t1 = cu[b + 1];
      t0 = t0 < 0 ? 0 : t0 > L ? L : t0;
      t1 = t1 < t0 ? t0 : t1 > L ? L : t1;
      len = t1 - t0;
      n = len <= seg ? 1 : (len - 1) / seg + 1;
    }
    long long x = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const long long up = __shfl_up(x, d, 64);
      if (lane >= d) x += up;
    }
    if (lane == 63) wsum[wave] = x;
    __syncthreads();
    long long before = base;
    for (int w = 0; w < wave; ++w) before += wsum[w];
    const long long total = wsum[0] + wsum[1] + wsum[2] + wsum[3];
    const long long at = before + x - n;
    if (b < B) {
      starts[b] = at < segs ? (int)at : segs;
      for (int i = 0; i < n; ++i) {
        // offsets that overlap could ask for more segments than their rows hold: those behind the bound are dropped
        if (at + i >= segs) break;
        int4 e;
        e.x = b;
        e.y = t0 + i * seg;
        e.z = len - i * seg < seg ? len - i * seg : seg;
        e.w = (i == 0 ? 1 : 0) | (i == n - 1 || at + i == segs - 1 ? 2 : 0);   // nothing is passed on behind the bound
        *(int4*)(table + 4 * (at + i)) = e;
      }
    }
    base += total;
    __syncthreads();
  }
  if (tid == 0) starts[B] = base < segs ? (int)base : segs;
  for (long long i = base + tid; i < segs; i += 256) *(int4*)(table + 4 * i) = make_int4(0, 0, -1, 0);
}

}  // namespace pdscan
