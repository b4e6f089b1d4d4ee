// Argument checks and workspace parts shared by the host side of the training operators
// (vb_train.cpp, vb_block.cpp).  Nothing here throws.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "vb_train_internal.h"

namespace vb {

inline vb_status fail(vb_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error(s, buf);
}

#define HIPCHK(expr)                                                                        \
  do {                                                                                      \
    hipError_t e_ = (expr);                                                                 \
    if (e_ != hipSuccess) return fail(VB_EDEVICE, "%s: %s", #expr, hipGetErrorString(e_)); \
  } while (0)

inline size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Bounds that keep byte offsets within a matrix below 2^62, row counts within a grid
// dimension and, for the layers, a row within MAX_CHUNKED_ROW bytes.
constexpr int64_t MAX_ROWS = 0x7fffffff, MAX_LD = INT64_C(1) << 30;
constexpr int32_t MAX_WIDTH = 1 << 20, MAX_CLASSES = 1 << 30;
static_assert(MAX_WIDTH * 4LL <= MAX_CHUNKED_ROW, "packed rows fit the product's offsets");

inline vb_status check_sizes(const char* fn, int64_t rows, int32_t n_in, int32_t n_out, int32_t dtype,
                             int32_t most = MAX_WIDTH) {
  if (rows < 0 || rows > MAX_ROWS) return fail(VB_EINVAL, "%s: rows must be in [0, 2^31) (got %lld)", fn, (long long)rows);
  if (n_in <= 0 || n_out <= 0) return fail(VB_EINVAL, "%s: sizes must be positive (got %d, %d)", fn, n_in, n_out);
  if (n_in > most || n_out > most)
    return fail(VB_EUNSUPPORTED, "%s: sizes above %d are not supported (got %d, %d)", fn, most, n_in, n_out);
  if (dtype < VB_F32 || dtype > VB_F16) return fail(VB_EINVAL, "%s: unknown dtype %d", fn, dtype);
  return VB_OK;
}

inline vb_status check_matrix(const char* fn, const char* name, const void* p, int64_t ld, int64_t n, int dtype, bool required,
                       int64_t most = MAX_LD) {
  if (!p) return required ? fail(VB_EINVAL, "%s: %s is NULL", fn, name) : VB_OK;
  if ((uintptr_t)p % elem_size(dtype)) return fail(VB_EINVAL, "%s: %s is not aligned to its elements", fn, name);
  if (ld < n || ld > most)
    return fail(VB_ESHAPE, "%s: leading dimension of %s must be in [%lld, 2^30] (got %lld)", fn, name, (long long)n, (long long)ld);
  return VB_OK;
}

inline vb_status check_ws(const char* fn, const void* ws, size_t ws_bytes, size_t need) {
  if (!need) return VB_OK;
  if (!ws || ws_bytes < need)
    return fail(VB_ENOMEM, "%s: workspace too small (%zu bytes, needs %zu)", fn, ws ? ws_bytes : (size_t)0, need);
  if ((uintptr_t)ws & 15) return fail(VB_EINVAL, "%s: workspace is not 16-byte aligned", fn);
  return VB_OK;
}

// An argument's memory, and whether the call writes it.
struct Named {
  const char* name;
  Span span;
  bool written;
};

inline Named matrix(const char* name, const void* p, int64_t rows, int64_t n, int64_t ld, int dtype, bool written) {
  const int64_t es = (int64_t)elem_size(dtype);
  return {name, {(uintptr_t)p, rows, n * es, ld * es}, written};
}

inline Named block(const char* name, const void* p, int64_t bytes, bool written) {
  return {name, {(uintptr_t)p, 1, bytes, bytes}, written};
}

// What is written shares no memory with anything else.  out: an output that may be the input
// `over`, or `over2`, itself (their pointers and leading dimensions are equal).
template <int N>
vb_status check_overlaps(const char* fn, const Named (&m)[N], int out = -1, int over = -1, int over2 = -1) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j) {
      if (!m[i].written || i == j || (m[j].written && j < i)) continue;
      if (i == out && (j == over || j == over2) && m[i].span.at == m[j].span.at) continue;
      if (overlap(m[i].span, m[j].span)) return fail(VB_EINVAL, "%s: %s overlaps %s", fn, m[i].name, m[j].name);
    }
  return VB_OK;
}

#define TRY(expr)                   \
  do {                              \
    if (vb_status s_ = (expr)) return s_; \
  } while (0)

// A part of the workspace: its offset, or none.
struct Part {
  size_t at = 0;
  bool used = false;
  void take(size_t& total, size_t bytes) {
    if (!bytes) return;
    at = total, used = true;
    total += align_up(bytes);
  }
  void* in(void* ws) const { return used ? (char*)ws + at : nullptr; }
};

// The products of a layer's backward pass, dx = g W and dweight = g^T x (vb_train.cpp).  g [rows]
// [n_g] is made in the workspace (make_g), in two parts where `two`, or is `given`.
struct BackwardCall {
  int64_t rows;
  int n_in, n_g, dtype;
  bool make_g;
  const void* given;
  int64_t ld_given;
  bool two;
  const void* x;
  int64_t ld_x;
  const void* weight;
  int64_t ld_w;
  void* dx;
  int64_t ld_dx;
  void* dweight;
  int64_t ld_dw;
  size_t sums_bytes;  // parts of dbias
};
struct BackwardPlan {
  Product dx{}, dw{};
  Part g, g_low, x, w, sums, partial, partial_w;  // partial_w: dw's, where both run at once
  Pair pair{};
  size_t total = 0;
};
BackwardPlan plan_backward(const BackwardCall& p);
// The copies of x and W that the products need.
PackJobs backward_copies(const BackwardCall& p, const BackwardPlan& f, void* ws);
// Both products, after g and the copies, and the last sums of dbias.
vb_status run_backward(const BackwardCall& p, BackwardPlan& f, const ColumnSums& sums, void* ws, hipStream_t st);

}  // namespace vb
