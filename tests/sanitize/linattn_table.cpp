// The segment-table kernel on the host, a thread for each of its 256 lanes:
// what it writes for offsets in order, and that offsets which ask for more
// segments than 32 bits count write nothing outside the table.
#include <barrier>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <thread>
#include <vector>

struct int4 {
  int x, y, z, w;
};
static int4 make_int4(int x, int y, int z, int w) { return int4{x, y, z, w}; }
static thread_local struct { unsigned x; } threadIdx;
static std::barrier<> g_barrier(256);
static void __syncthreads() { g_barrier.arrive_and_wait(); }
template <typename T>
static T __shfl_up(T x, unsigned d, int) {
  static T lane_value[256];
  lane_value[threadIdx.x] = x;
  __syncthreads();
  const unsigned lane = threadIdx.x & 63;
  const T y = lane >= d ? lane_value[threadIdx.x - d] : x;
  __syncthreads();
  return y;
}
#define __global__
#define __launch_bounds__(n)
#define __shared__ static

#include "pdscan_linattn_table.h"

static int g_fail = 0;

static void check(bool ok, const char* what) {
  if (!ok) {
    std::fprintf(stderr, "FAIL %s\n", what);
    ++g_fail;
  }
}

struct Result {
  std::vector<int32_t> table, starts;
  bool clean;   // the guards around both are as they were
};

static Result table_of(const std::vector<int32_t>& cu, int L, int seg, int segs) {
  constexpr int G = 4096;
  const int B = (int)cu.size() - 1;
  std::vector<int32_t> t(4 * (size_t)segs + 2 * G, 77), s(B + 1 + 2 * G, 77);
  std::vector<std::thread> lanes;
  for (unsigned i = 0; i < 256; ++i)
    lanes.emplace_back([&, i] {
      threadIdx.x = i;
      pdscan::pdssm_linattn_table_kernel(cu.data(), t.data() + G, s.data() + G, B, L, seg, segs);
    });
  for (auto& l : lanes) l.join();
  Result r;
  r.table.assign(t.begin() + G, t.end() - G);
  r.starts.assign(s.begin() + G, s.end() - G);
  r.clean = true;
  for (int i = 0; i < G; ++i)
    if (t[i] != 77 || t[t.size() - 1 - i] != 77 || s[i] != 77 || s[s.size() - 1 - i] != 77) r.clean = false;
  return r;
}

// Every entry lies in the rows, and the starts rise within the table.
static void sound(const Result& r, int L, int seg, int segs, const char* what) {
  check(r.clean, what);
  for (int i = 0; i < segs; ++i) {
    const int32_t* e = &r.table[4 * (size_t)i];
    if (e[2] < 0) continue;
    check(e[0] >= 0 && e[0] < (int)r.starts.size() - 1 && e[1] >= 0 && e[2] <= seg && (int64_t)e[1] + e[2] <= L, what);
  }
  for (size_t b = 0; b < r.starts.size(); ++b)
    check(r.starts[b] >= (b ? r.starts[b - 1] : 0) && r.starts[b] <= segs, what);
}

int main() {
  {   // in order, with empty sequences, more than one round of 256
    std::vector<int32_t> cu(1, 0);
    for (int b = 0; b < 300; ++b) cu.push_back(cu.back() + (b % 7 == 0 ? 0 : b % 50 == 1 ? 200 : 3));
    const int L = cu.back() + 5, seg = 64, segs = L / seg + 300;
    const Result r = table_of(cu, L, seg, segs);
    sound(r, L, seg, segs, "in order");
    int at = 0;
    for (int b = 0; b < 300; ++b) {
      check(r.starts[b] == at, "start");
      const int len = cu[b + 1] - cu[b], n = len <= seg ? 1 : (len - 1) / seg + 1;
      for (int i = 0; i < n; ++i, ++at) {
        const int32_t* e = &r.table[4 * (size_t)at];
        check(e[0] == b && e[1] == cu[b] + i * seg && e[2] == (len - i * seg < seg ? len - i * seg : seg) &&
                  e[3] == ((i == 0) | (i == n - 1) << 1),
              "entry");
      }
    }
    check(r.starts[300] == at, "end");
    for (; at < segs; ++at) check(r.table[4 * (size_t)at + 2] == -1, "behind the last");
  }
  // offsets up and down: every other sequence spans all rows
  for (int L : {1 << 20, 0x7fffff00})
    for (int B : {70, 300, 1000}) {
      std::vector<int32_t> cu;
      for (int b = 0; b <= B; ++b) cu.push_back(b & 1 ? L : 0);
      sound(table_of(cu, L, 64, 1000), L, 64, 1000, "up and down");
    }
  {   // far below and above the rows
    std::vector<int32_t> cu;
    for (int b = 0; b <= 600; ++b) cu.push_back(b & 1 ? 0x7fffffff : (int32_t)0x80000000);
    sound(table_of(cu, 0x7fffff00, 512, 64), 0x7fffff00, 512, 64, "ends of 32 bits");
  }
  std::printf("ok: %d failures\n", g_fail);
  return g_fail != 0;
}
