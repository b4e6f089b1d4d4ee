// The test for shared bytes of two matrices (vb_train_internal.h) against marking them one by
// one, over every small shape and many random ones.  Exit status 0 when they agree.
#include <cstdio>
#include <random>
#include <vector>

#include "vb_train_internal.h"

namespace {

bool marked(const vb::Span& a, const vb::Span& b) {
  std::vector<char> m(4096, 0);
  for (int64_t r = 0; r < a.rows; ++r)
    for (int64_t i = 0; i < a.bytes; ++i) m[a.at + r * a.ld + i] = 1;
  for (int64_t r = 0; r < b.rows; ++r)
    for (int64_t i = 0; i < b.bytes; ++i)
      if (m[b.at + r * b.ld + i]) return true;
  return false;
}

}  // namespace

int main() {
  std::mt19937 rng(7);
  auto up_to = [&](int n) { return (int64_t)(rng() % n); };
  long long checks = 0, failures = 0, shared = 0;
  auto check = [&](const vb::Span& a, const vb::Span& b) {
    const bool want = marked(a, b);
    ++checks, shared += want;
    if (vb::overlap(a, b) != want || vb::overlap(b, a) != want) {
      if (++failures < 10)
        std::printf("FAIL %lld+%lldx%lld/%lld %lld+%lldx%lld/%lld: %d\n", (long long)a.at, (long long)a.rows, (long long)a.bytes,
                    (long long)a.ld, (long long)b.at, (long long)b.rows, (long long)b.bytes, (long long)b.ld, want);
    }
  };
  for (int i = 0; i < 400000; ++i) {
    vb::Span a{(uintptr_t)(1 + up_to(60)), up_to(6), up_to(9), 0}, b{(uintptr_t)(1 + up_to(60)), up_to(6), up_to(9), 0};
    a.ld = a.bytes + up_to(12), b.ld = i % 2 ? b.bytes + up_to(12) : a.ld;
    if (b.ld < b.bytes) b.bytes = b.ld;
    check(a, b);
  }
  // two ranges of columns of one buffer, and the same a byte too wide
  const vb::Span left{1000, 50, 24, 40};
  check(left, {1024, 50, 16, 40});
  check(left, {1023, 50, 16, 40});
  check(left, {1024, 50, 17, 40});
  // large ones, which are not marked: rows 2^31 apart, and the largest that the calls take
  const int64_t rows = 0x7fffffff, ld = INT64_C(1) << 32;
  const vb::Span x{4096, rows, 1 << 20, ld}, y{4096 + (1 << 20), rows, 1 << 20, ld}, z{4096 + (1 << 20) - 1, rows, 1 << 20, ld};
  checks += 3;
  if (vb::overlap(x, y) || !vb::overlap(x, z) || !vb::overlap(z, y)) std::printf("FAIL large\n"), ++failures;
  std::printf("%lld checks, %lld of them shared, %lld failure(s)\n", checks, shared, failures);
  return failures != 0;
}
