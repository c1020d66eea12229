// Every unit of a scan's launch belongs to one workgroup, also where the grid
// takes several rows, the last of which may reach behind the units.
#include <cstdio>
#include <vector>

#include "pdscan_ssm_plan.h"

int main() {
  int failures = 0;
  const long long row = 0xffffffffll / 256;   // workgroups of 256 threads in one row
  for (long long n : {1ll, 7ll, 8ll, 9ll, 1000ll, row - 1, row, row + 1, 2 * row + 9, 3 * row + 17, 5 * row + 3, 7 * row + 1}) {
    const pdscan::LaGrid g = pdscan::la_grid_rows((n + 7) / 8 * 8, 256);
    std::vector<unsigned char> seen((size_t)n, 0);
    long long twice = 0, missing = 0;
    for (long long id = 0; id < (long long)g.x * g.y; ++id) {
      const long long u = pdscan::ss_near((unsigned)id, n);
      if (u < 0) ++twice;
      else if (u < n && seen[(size_t)u]++) ++twice;
    }
    for (unsigned char c : seen) missing += !c;
    if (twice || missing) {
      std::fprintf(stderr, "FAIL %lld units: %lld taken twice, %lld not at all\n", n, twice, missing);
      ++failures;
    }
  }
  std::printf("ok: %d failures\n", failures);
  return failures != 0;
}
