// Host-side checks of the training operators' C ABI (vb_train.h), built with
// AddressSanitizer and UndefinedBehaviorSanitizer around the library's host code.  Every
// call here sizes a workspace or is rejected before anything is enqueued; device
// pointers are fake addresses that are never read.  Exit status 0 when every call
// returned what is expected.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

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

vb_linear_fwd forward(int64_t rows, int32_t n_in, int32_t n_out, int32_t dtype, uintptr_t at) {
  vb_linear_fwd p{};
  p.rows = rows, p.n_in = n_in, p.n_out = n_out, p.dtype = dtype;
  p.x = fake(at), p.ld_x = n_in, p.weight = fake(at), p.ld_w = n_in;
  p.y = fake(4096), p.ld_y = n_out;
  return p;
}

vb_linear_bwd backward(int64_t rows, int32_t n_in, int32_t n_out, int32_t dtype, uintptr_t at) {
  vb_linear_bwd p{};
  p.rows = rows, p.n_in = n_in, p.n_out = n_out, p.dtype = dtype, p.act = VB_ACT_GELU;
  p.dy = p.saved = fake(at), p.ld_dy = p.ld_saved = n_out;
  p.x = fake(at), p.ld_x = n_in, p.weight = fake(at), p.ld_w = n_in;
  p.dx = p.dweight = p.dbias = p.dresidual = fake(4096);
  p.ld_dx = p.ld_dw = n_in, p.ld_dres = n_out;
  return p;
}

}  // namespace

int main() {
  // workspaces over the whole range of sizes, and the calls with a byte too little
  const int32_t widths[] = {1, 7, 8, 100, 784, 1023, 4096, 65537, 1 << 20};
  const int64_t rows[] = {0, 1, 16, 33, 1000, 65536, 2147483647};
  for (int32_t dtype = 0; dtype < 3; ++dtype)
    for (int64_t m : rows)
      for (int32_t k : widths)
        for (int32_t n : widths)
          for (uintptr_t at : {uintptr_t(4096), uintptr_t(4100)}) {
            size_t need = 0;
            const vb_linear_fwd f = forward(m, k, n, dtype, at);
            expect(vb_linear_forward_workspace(&f, &need) == VB_OK, "forward workspace");
            if (m && need) expect(vb_linear_forward(&f, fake(4096), need - 1, nullptr) == VB_ENOMEM, "short workspace");
            const vb_linear_bwd b = backward(m, k, n, dtype, at);
            expect(vb_linear_backward_workspace(&b, &need) == VB_OK, "backward workspace");
            expect(m == 0 ? need == 0 : need >= (size_t)m * n * (dtype ? 2 : 4), "backward workspace holds g");
            if (m) expect(vb_linear_backward(&b, fake(4096), need - 1, nullptr) == VB_ENOMEM, "short workspace");
          }
  size_t need = 0;
  vb_linear_fwd f = forward(8, (1 << 20) + 1, 8, 0, 4096);
  expect(vb_linear_forward_workspace(&f, &need) == VB_EUNSUPPORTED, "too wide");
  f = forward(8, 8, INT32_MAX, 0, 4096);
  expect(vb_linear_forward(&f, nullptr, 0, nullptr) == VB_EUNSUPPORTED, "too wide");
  f = forward(INT64_MIN, 8, 8, 0, 4096);
  expect(vb_linear_forward(&f, nullptr, 0, nullptr) == VB_EINVAL, "negative rows");
  f = forward(8, 8, 8, 0, 4096);
  f.ld_x = INT64_MAX;
  expect(vb_linear_forward(&f, nullptr, 0, nullptr) == VB_ESHAPE, "leading dimension");

  for (int64_t m : rows) {
    expect(vb_cross_entropy_workspace(m, 1 << 30, VB_F32, &need) == VB_OK && need >= (size_t)m * 4, "loss workspace");
    vb_cross_entropy_args a{};
    a.rows = m, a.classes = 10, a.logits = fake(4096), a.ld = 10, a.labels = (const int64_t*)fake(4096);
    a.loss = (float*)fake(4096);
    expect(vb_cross_entropy(&a, fake(4096), 8, nullptr) == VB_ENOMEM, "short loss workspace");
  }
  expect(vb_cross_entropy_workspace(8, INT32_MAX, VB_F32, &need) == VB_EUNSUPPORTED, "too many classes");

  std::vector<int64_t> sizes(1000, 100003);
  std::vector<const void*> grads(sizes.size(), fake(4096));
  std::vector<int32_t> types(sizes.size(), VB_BF16);
  expect(vb_clip_grad_norm_workspace((int32_t)sizes.size(), sizes.data(), &need) == VB_OK, "clip workspace");
  expect(vb_clip_grad_norm((int32_t)sizes.size(), grads.data(), nullptr, sizes.data(), types.data(), 1.f,
                           (float*)fake(4096), fake(4096), need - 1, nullptr) == VB_ENOMEM, "short clip workspace");
  types.back() = 7;
  expect(vb_clip_grad_norm((int32_t)sizes.size(), grads.data(), nullptr, sizes.data(), types.data(), 1.f,
                           (float*)fake(4096), fake(4096), need, nullptr) == VB_EINVAL && std::strstr(vb_last_error(), "999"),
         "type of the last tensor");
  sizes[3] = INT64_MAX;
  expect(vb_clip_grad_norm_workspace((int32_t)sizes.size(), sizes.data(), &need) == VB_EINVAL, "a size too large");
  sizes.assign(sizes.size(), INT64_C(1) << 43);
  expect(vb_clip_grad_norm_workspace((int32_t)sizes.size(), sizes.data(), &need) == VB_EINVAL, "a total too large");
  std::printf("%d checks, %d failure(s)\n", checks, failures);
  return failures != 0;
}
