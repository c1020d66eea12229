// The grids of the largest calls: what passes the checks fits the device, and
// what does not is refused before the first launch.
#include "linattn_stubs.h"

static void passes(int (*call)(const pdssm_linattn_dims&), const pdssm_linattn_dims& d, const char* what) {
  expect(call(d), PDSSM_OK, what);
}
static void refused(int (*call)(const pdssm_linattn_dims&), const pdssm_linattn_dims& d, const char* what) {
  const int launches = g_launches;
  expect(call(d), PDSSM_EUNSUPPORTED, what);
  expect(g_launches - launches, 0, what);
}

int main() {
  // one row of workgroups up to 2^32 - 1 threads, then more
  const pdscan::LaGrid one = pdscan::la_grid_rows((1 << 23) - 1, 512), two = pdscan::la_grid_rows(1 << 23, 512);
  if (one.x != (1 << 23) - 1 || one.y != 1 || two.x != 1 << 22 || two.y != 2) ++g_fail;
  // sequences of one token: the log-decay gradient has 512 threads a sequence and head
  passes(call_bwd, dims(262143, 32, 32, 1, 8, 8), "gradient of one row");
  passes(call_bwd, dims(262144, 32, 32, 1, 8, 8), "gradient of two rows");
  passes(call_bwd, dims(1 << 22, 1, 1, 1, 256, 256), "gradient, wide rows");
  passes(call_bwd, dims(1 << 22, 32, 32, 1 << 22, 8, 8, 1), "gradient, packed");
  passes(call_fwd, dims(1 << 26, 1, 1, 1, 8, 8), "forward of two rows");
  passes(call_fwd, dims(1 << 23, 1, 1, 1, 8, 256), "forward, two slabs");
  passes(call_step, dims((1 << 24) + 1, 1, 1, 1, 8, 8), "step of two rows");
  passes(call_step, dims(0x7fffffff, 1, 1, 1, 8, 8), "the largest step");
  refused(call_fwd, dims(0x7fffffff, 1, 1, 1, 8, 8), "forward, workgroups past 31 bits");
  refused(call_bwd, dims(1 << 24, 1 << 5, 1, 1, 8, 8), "gradient, workgroups past 31 bits");
  // every size that passes, around the powers of two, batched and packed
  long long calls = 0;
  for (int lb = 0; lb <= 27; lb += 3)
    for (int off = -1; off <= 1; ++off)
      for (int H : {1, 6, 1 << 10})
        for (int L : {1, 300, 100000})
          for (int dk : {8, 64, 136})
            for (int dv : {32, 256})
              for (int packed = 0; packed < 2; ++packed)
                for (int dtype : {PDSSM_F32, PDSSM_BF16}) {
                  const int B = (1 << lb) + off;
                  if (B < 1) continue;
                  const pdssm_linattn_dims d = dims(B, H, H, L, dk, dv, packed, dtype);
                  const int before = g_launches, rf = call_fwd(d);
                  if (rf != PDSSM_OK && g_launches != before) ++g_fail;
                  const int between = g_launches, rb = call_bwd(d);
                  if (rb != PDSSM_OK && g_launches != between) ++g_fail;
                  calls += 2;
                }
  std::printf("ok: %d failures, %lld calls, %d launches\n", g_fail, calls, g_launches);
  return g_fail != 0;
}
