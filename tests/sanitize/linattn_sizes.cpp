// Workspace queries of the linear-attention calls at the largest sizes that
// their arguments can name: each is answered or refused, with no overflow on
// the way.
#include "linattn_stubs.h"

int main() {
  const int big[] = {1, 2, 3, 1 << 20, 1 << 28, 1 << 29, 0x2aaaaaab, 1 << 30, 0x55555556, 0x7fffff00, 0x7fffffff};
  const int small[] = {1, 2, 255, 1 << 16, 0x7fffffff};
  const int lengths[] = {1, 256, 257, 1 << 20, 0x7fffff00, 0x7fffffff};
  const int wide[] = {8, 32, 72, 136, 256};
  long long asked = 0;
  for (int H : big)
    for (int B : small)
      for (int L : lengths)
        for (int dk : wide)
          for (int dv : wide)
            for (int packed = 0; packed < 2; ++packed)
              for (int dtype : {PDSSM_F32, PDSSM_BF16}) {
                const pdssm_linattn_dims d = dims(B, H, H, L, dk, dv, packed, dtype);
                size_t f = 0, b = 0;
                const int rf = pdssm_linattn_workspace_bytes(&d, &f), rb = pdssm_linattn_bwd_workspace_bytes(&d, &b);
                if (rf != PDSSM_OK && rf != PDSSM_EUNSUPPORTED) ++g_fail;
                if (rb != PDSSM_OK && rb != PDSSM_EUNSUPPORTED) ++g_fail;
                if (rf == PDSSM_OK && f < 256) ++g_fail;
                if (rb == PDSSM_OK && b < 256) ++g_fail;
                asked += 2;
              }
  size_t n = 0;
  // heads times jobs times column slabs is 2^32 and more
  pdssm_linattn_dims d = dims(1, 1 << 30, 1 << 30, 1, 256, 8);
  expect(pdssm_linattn_bwd_workspace_bytes(&d, &n), PDSSM_EUNSUPPORTED, "2^30 heads, gradient");
  d = dims(1, 0x7fffffff, 0x7fffffff, 1, 8, 256);
  expect(pdssm_linattn_workspace_bytes(&d, &n), PDSSM_EUNSUPPORTED, "2^31 - 1 heads of two slabs");
  expect(pdssm_linattn_bwd_workspace_bytes(&d, &n), PDSSM_EUNSUPPORTED, "2^31 - 1 heads of two slabs, gradient");
  std::printf("ok: %d failures, %lld queries\n", g_fail, asked);
  return g_fail != 0;
}
