// The tiles that a layer's backward pass chooses for both of its products (vb_train_internal.h).
// Exit status 0 when they are as they should be.
#include <cstdio>

#include "vb_train_internal.h"

namespace {

int failures = 0, checks = 0;

vb::Pair pair_of(long long rows, int n_in, int n_g, int dtype, int passes) {
  vb::Product dx{}, dw{};
  dx.passes = dw.passes = passes;
  dx.across_b = dw.across_a = dw.across_b = true;
  dx.M = rows, dx.N = n_in, dx.K = n_g;
  dw.M = n_g, dw.N = n_in, dw.K = rows;
  return vb::choose_pair(dx, dw, dtype);
}

void expect(bool ok, const char* what, long long rows, int n_in, int n_g, vb::Pair p) {
  ++checks;
  if (ok) return;
  std::printf("FAIL %s: %lld x %d -> %d: tiles of %d, %d and %d parts\n", what, rows, n_in, n_g, p.tile, p.splits_x, p.splits_w);
  ++failures;
}

}  // namespace

int main() {
  // float32, a reduction split: 64-wide tiles or launches of their own
  const int sizes[] = {1, 7, 28, 100, 377, 622, 1121, 1243, 2097, 4848, 8192, 14556};
  for (int rows : sizes)
    for (int n_in : sizes)
      for (int n_g : sizes) {
        const vb::Pair p = pair_of(rows, n_in, n_g, VB_F32, 1);
        expect(p.tile <= 64 || (p.splits_x == 1 && p.splits_w == 1), "wide tiles of a split reduction", rows, n_in, n_g, p);
      }
  // small split reductions share a launch, in every type
  for (int dtype = VB_F32; dtype <= VB_F16; ++dtype) {
    vb::Pair p = pair_of(28, 26, 926, dtype, 1);
    expect(p.tile == 64 && p.splits_x > 1, "a small pair", 28, 26, 926, p);
    p = pair_of(728, 49, 780, dtype, dtype == VB_F32 ? 1 : 2);
    expect(p.tile == 64 && p.splits_x > 1 && p.splits_w > 1, "a small pair", 728, 49, 780, p);
  }
  std::printf("%d checks, %d failure(s)\n", checks, failures);
  return failures != 0;
}
