// Host-side checks of the C ABI of the gated linear layer, layer norm and dropout
// (vb_train.h), built with AddressSanitizer and UndefinedBehaviorSanitizer around the
// library's host code.  Every call here sizes a workspace or is rejected before anything is
// enqueued; device pointers are fake addresses that are never read.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "vb_train.h"

namespace {

int failures = 0, checks = 0;

void expect(bool ok, const char* what) {
  ++checks;
  if (!ok) {
    std::printf("FAIL %s: '%s'\n", what, vb_last_error());
    ++failures;
  }
}

void* fake(uintptr_t a) { return reinterpret_cast<void*>(a); }

}  // namespace

int main() {
  const int32_t widths[] = {1, 7, 8, 100, 784, 1023, 4096, 65537, 1 << 19, 1 << 20};
  const int64_t rows[] = {0, 1, 16, 33, 1000, 65536, 2147483647};
  for (int32_t dtype = 0; dtype < 3; ++dtype)
    for (int64_t m : rows)
      for (int32_t k : widths) {
        size_t need = 0;
        for (int32_t n : widths)
          for (uintptr_t at : {uintptr_t(4096), uintptr_t(4100)}) {
            vb_gated_linear_fwd f{};
            f.rows = m, f.n_in = k, f.n_out = n, f.dtype = dtype;
            f.x = f.weight = fake(at), f.ld_x = f.ld_w = k, f.y = fake(4096), f.ld_y = n;
            vb_gated_linear_bwd b{};
            b.rows = m, b.n_in = k, b.n_out = n, b.dtype = dtype;
            b.dy = b.pre = b.x = b.weight = fake(at), b.ld_dy = n, b.ld_pre = 2 * (int64_t)n, b.ld_x = b.ld_w = k;
            b.dx = b.dweight = b.dbias = fake(4096), b.ld_dx = b.ld_dw = k;
            if (n > 1 << 19) {
              expect(vb_gated_linear_forward_workspace(&f, &need) == VB_EUNSUPPORTED, "too wide");
              expect(vb_gated_linear_backward(&b, nullptr, 0, nullptr) == VB_EUNSUPPORTED, "too wide");
              continue;
            }
            expect(vb_gated_linear_forward_workspace(&f, &need) == VB_OK, "forward workspace");
            if (m && need) expect(vb_gated_linear_forward(&f, fake(4096), need - 1, nullptr) == VB_ENOMEM, "short workspace");
            expect(vb_gated_linear_backward_workspace(&b, &need) == VB_OK, "backward workspace");
            expect(m == 0 ? need == 0 : need >= 2 * (size_t)m * n * (dtype ? 2 : 4), "backward workspace holds g");
            if (m) expect(vb_gated_linear_backward(&b, fake(4096), need - 1, nullptr) == VB_ENOMEM, "short workspace");
          }
        expect(vb_layer_norm_backward_workspace(m, k, dtype, &need) == VB_OK, "norm workspace");
        vb_layer_norm_bwd g{};
        g.rows = m, g.n = k, g.dtype = dtype;
        g.dy = g.x = fake(4096), g.mean = g.rstd = (const float*)fake(4096), g.ld_dy = g.ld_x = k;
        g.dweight = fake(4096);
        if (m) expect(need >= 8 * (size_t)k && vb_layer_norm_backward(&g, fake(4096), need - 1, nullptr) == VB_ENOMEM, "short workspace");
        vb_dropout_args d{};
        d.rows = m, d.n = k, d.dtype = dtype, d.x = fake(4096), d.y = fake(4096 + 2 + (dtype ? 0 : 2)), d.ld_x = d.ld_y = k, d.p = 0.5;
        if (m > 1 || (m && k > 1)) expect(vb_dropout(&d, nullptr) == VB_EINVAL, "overlapping output");
        d.p = NAN;
        expect(vb_dropout(&d, nullptr) == VB_EINVAL, "p");
        vb_layer_norm_fwd l{};
        l.rows = m, l.n = k, l.dtype = dtype, l.eps = -1.f;
        expect(vb_layer_norm_forward(&l, nullptr) == VB_EINVAL, "eps");
      }
  vb_dropout_args d{};
  d.rows = INT64_MIN, d.n = INT32_MAX;
  expect(vb_dropout(&d, nullptr) < 0, "rows");
  d.rows = 2147483647, d.n = 1 << 30, d.x = fake(4096), d.ld_x = INT64_MAX;
  expect(vb_dropout(&d, nullptr) == VB_ESHAPE, "leading dimension");
  std::printf("%d checks, %d failure(s)\n", checks, failures);
  return failures != 0;
}
