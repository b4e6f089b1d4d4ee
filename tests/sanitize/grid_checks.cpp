// The grids of large launches (vb_train_internal.h) stay within what a launch may hold and
// cover every workgroup once.  Exit status 0 when they do.
#include <cstdio>

#include "vb_train_internal.h"

int main() {
  int failures = 0, checks = 0;
  const long long last = 1LL << 31;
  for (long long around : {1LL, 2LL, 255LL, 4096LL, 1LL << 20, 1LL << 21, 1LL << 22, 1LL << 24, 1LL << 26, 1LL << 30, last})
    for (long long blocks = around - 9; blocks <= around + 9; ++blocks)
      for (unsigned y : {1u, 32u}) {
        if (blocks < 1 || blocks > last) continue;
        const dim3 g = vb::grid_of(blocks, y);
        const long long all = (long long)g.x * g.z;
        bool ok = g.y == y && g.x >= 1 && g.z >= 1 && g.z <= 65535 && (long long)g.x * 1024 < 1LL << 32;
        ok = ok && all >= blocks && all - blocks < g.x && all <= 1LL << 32;
        ok = ok && (g.z == 1 ? g.x == blocks : g.x == vb::GRID_X);  // workgroup_number counts in steps of GRID_X
        ++checks;
        if (!ok) {
          std::printf("FAIL %lld blocks: %u x %u x %u\n", blocks, g.x, g.y, g.z);
          ++failures;
        }
      }
  static_assert(vb::CLIP_MAX_CHUNKS * 256 < 1LL << 32, "a launch over all chunks of a call");
  std::printf("%d checks, %d failure(s)\n", checks, failures);
  return failures != 0;
}
