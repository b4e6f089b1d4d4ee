// C ABI of the training operators (include/vb_train.h): argument checks and the
// sequence of launches.  Nothing here throws.
#include <algorithm>
#include <cmath>
#include <new>

#include "vb_train.h"
#include "vb_train_host.h"

using namespace vb;

namespace {

// The forward product, and copies of operands whose rows a large product cannot read.
struct ForwardPlan {
  Product d{};
  Part x, w, partial;
  size_t total = 0;
};

ForwardPlan plan_forward(const vb_linear_fwd& p) {
  ForwardPlan f;
  Product& d = f.d;
  d.a = p.x, d.lda = p.ld_x;
  d.b = p.weight, d.ldb = p.ld_w;
  d.M = p.rows, d.N = p.n_out, d.K = p.n_in, d.passes = 1;
  d.bias = p.bias, d.res = p.residual, d.ld_res = p.ld_res;
  d.out = p.y, d.ld_out = p.ld_y, d.pre = p.pre, d.ld_pre = p.ld_pre, d.act = p.act;
  if (p.rows == 0 || product_is_narrow(d, p.dtype)) return f;
  const size_t row = chunked_row(p.n_in, p.dtype);
  if (!is_chunked(p.x, p.ld_x, p.n_in, p.dtype)) f.x.take(f.total, p.rows * row);
  if (!is_chunked(p.weight, p.ld_w, p.n_in, p.dtype)) f.w.take(f.total, p.n_out * row);
  f.partial.take(f.total, product_bytes(d, p.dtype));
  return f;
}

// g is dy itself without an activation, else (or if dy's rows cannot be read by a large
// product) a copy, in two parts where one number of the type does not hold it.
BackwardCall backward_call(const vb_linear_bwd& p) {
  BackwardCall c{};
  c.rows = p.rows, c.n_in = p.n_in, c.n_g = p.n_out, c.dtype = p.dtype;
  c.make_g = p.act != VB_ACT_NONE || !is_chunked(p.dy, p.ld_dy, p.n_out, p.dtype);
  c.given = p.dy, c.ld_given = p.ld_dy;
  c.two = p.dtype != VB_F32 && (p.act == VB_ACT_GELU || p.act == VB_ACT_SILU) && !p.round_g;
  c.x = p.x, c.ld_x = p.ld_x, c.weight = p.weight, c.ld_w = p.ld_w;
  c.dx = p.dx, c.ld_dx = p.ld_dx, c.dweight = p.dweight, c.ld_dw = p.ld_dw;
  if (p.dbias && p.rows > 0) c.sums_bytes = act_grad_bytes(p.rows, p.n_out, p.dtype);
  return c;
}

}  // namespace

BackwardPlan vb::plan_backward(const BackwardCall& p) {
  BackwardPlan f;
  if (p.rows == 0) return f;
  const int dt = p.dtype;
  const long long ld_g = (long long)(chunked_row(p.n_g, dt) / elem_size(dt));
  Product& a = f.dx;
  a.a = p.given, a.lda = p.make_g ? ld_g : p.ld_given;
  a.b = p.weight, a.ldb = p.ld_w, a.across_b = true;
  a.M = p.rows, a.N = p.n_in, a.K = p.n_g;
  a.out = p.dx, a.ld_out = p.ld_dx;
  Product& b = f.dw;
  b.a = a.a, b.lda = a.lda, b.across_a = true;
  b.b = p.x, b.ldb = p.ld_x, b.across_b = true;
  b.M = p.n_g, b.N = p.n_in, b.K = p.rows;
  b.out = p.dweight, b.ld_out = p.ld_dw;
  a.passes = b.passes = p.two ? 2 : 1;
  if ((p.dx || p.dweight) && p.make_g) {
    f.g.take(f.total, p.rows * chunked_row(p.n_g, dt));
    if (p.two) f.g_low.take(f.total, p.rows * chunked_row(p.n_g, dt));
  }
  const size_t row = chunked_row(p.n_in, dt);
  if (p.dweight && !is_chunked(p.x, p.ld_x, p.n_in, dt)) f.x.take(f.total, p.rows * row);
  if (p.dx && !is_chunked(p.weight, p.ld_w, p.n_in, dt)) f.w.take(f.total, p.n_g * row);
  f.sums.take(f.total, p.sums_bytes);
  if (p.dx && p.dweight) f.pair = choose_pair(a, b, dt);
  if (f.pair.tile) {
    f.partial.take(f.total, pair_bytes(f.pair, a, f.pair.splits_x));
    f.partial_w.take(f.total, pair_bytes(f.pair, b, f.pair.splits_w));
    return f;
  }
  size_t parts = 0;  // the products run one after the other
  if (p.dx) parts = product_bytes(a, dt);
  if (p.dweight) {
    const size_t q = product_bytes(b, dt);
    if (q > parts) parts = q;
  }
  f.partial.take(f.total, parts);
  return f;
}

PackJobs vb::backward_copies(const BackwardCall& p, const BackwardPlan& f, void* ws) {
  return {{{p.x, p.ld_x, p.rows, p.n_in, f.x.in(ws)}, {p.weight, p.ld_w, p.n_g, p.n_in, f.w.in(ws)}}};
}

vb_status vb::run_backward(const BackwardCall& p, BackwardPlan& f, const ColumnSums& sums, void* ws, hipStream_t st) {
  if (f.g.used) f.dx.a = f.dw.a = f.g.in(ws), f.dx.a_low = f.dw.a_low = f.g_low.in(ws);
  const long long ld = (long long)(chunked_row(p.n_in, p.dtype) / elem_size(p.dtype));
  if (f.w.used) f.dx.b = f.w.in(ws), f.dx.ldb = ld;
  if (f.x.used) f.dw.b = f.x.in(ws), f.dw.ldb = ld;
  f.dx.partial = f.dw.partial = (float*)f.partial.in(ws);
  if (f.pair.tile) {
    f.dw.partial = (float*)f.partial_w.in(ws);
    HIPCHK(launch_pair(f.dx, f.dw, f.pair, sums, p.dtype, st));
    return VB_OK;
  }
  if (sums.out) HIPCHK(launch_column_sums(sums, p.dtype, st));
  if (p.dx) HIPCHK(launch_product(f.dx, p.dtype, st));
  if (p.dweight) HIPCHK(launch_product(f.dw, p.dtype, st));
  return VB_OK;
}

extern "C" vb_status vb_linear_forward_workspace(const vb_linear_fwd* p, size_t* bytes) {
  const char* fn = "vb_linear_forward_workspace";
  if (!p || !bytes) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_sizes(fn, p->rows, p->n_in, p->n_out, p->dtype));
  *bytes = plan_forward(*p).total;
  return VB_OK;
}

extern "C" vb_status vb_linear_backward_workspace(const vb_linear_bwd* p, size_t* bytes) {
  const char* fn = "vb_linear_backward_workspace";
  if (!p || !bytes) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_sizes(fn, p->rows, p->n_in, p->n_out, p->dtype));
  *bytes = plan_backward(backward_call(*p)).total;
  return VB_OK;
}

extern "C" vb_status vb_linear_forward(const vb_linear_fwd* p, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "vb_linear_forward";
  if (!p) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_sizes(fn, p->rows, p->n_in, p->n_out, p->dtype));
  if (p->act < VB_ACT_NONE || p->act > VB_ACT_SILU) return fail(VB_EINVAL, "%s: unknown activation %d", fn, p->act);
  if (p->rows == 0) return VB_OK;
  TRY(check_matrix(fn, "x", p->x, p->ld_x, p->n_in, p->dtype, true));
  TRY(check_matrix(fn, "weight", p->weight, p->ld_w, p->n_in, p->dtype, true));
  TRY(check_matrix(fn, "bias", p->bias, p->n_out, p->n_out, p->dtype, false));
  TRY(check_matrix(fn, "residual", p->residual, p->ld_res, p->n_out, p->dtype, false));
  TRY(check_matrix(fn, "y", p->y, p->ld_y, p->n_out, p->dtype, true));
  TRY(check_matrix(fn, "pre", p->pre, p->ld_pre, p->n_out, p->dtype, false));
  if (p->residual == p->y && p->ld_res != p->ld_y) return fail(VB_ESHAPE, "%s: y over residual needs the same leading dimension", fn);
  ForwardPlan f = plan_forward(*p);
  TRY(check_ws(fn, ws, ws_bytes, f.total));
  const Named memory[] = {matrix("y", p->y, p->rows, p->n_out, p->ld_y, p->dtype, true),
                          matrix("pre", p->pre, p->rows, p->n_out, p->ld_pre, p->dtype, true),
                          block("the workspace", ws, (int64_t)f.total, true),
                          matrix("residual", p->residual, p->rows, p->n_out, p->ld_res, p->dtype, false),
                          matrix("x", p->x, p->rows, p->n_in, p->ld_x, p->dtype, false),
                          matrix("weight", p->weight, p->n_out, p->n_in, p->ld_w, p->dtype, false),
                          matrix("bias", p->bias, 1, p->n_out, p->n_out, p->dtype, false)};
  TRY(check_overlaps(fn, memory, 0, 3));
  const hipStream_t st = (hipStream_t)stream;
  const long long ld = (long long)(chunked_row(p->n_in, p->dtype) / elem_size(p->dtype));
  HIPCHK(launch_pack({{{p->x, p->ld_x, p->rows, p->n_in, f.x.in(ws)}, {p->weight, p->ld_w, p->n_out, p->n_in, f.w.in(ws)}}},
                     p->dtype, st));
  if (f.x.used) f.d.a = f.x.in(ws), f.d.lda = ld;
  if (f.w.used) f.d.b = f.w.in(ws), f.d.ldb = ld;
  f.d.partial = (float*)f.partial.in(ws);
  HIPCHK(launch_product(f.d, p->dtype, st));
  return VB_OK;
}

extern "C" vb_status vb_linear_backward(const vb_linear_bwd* p, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "vb_linear_backward";
  if (!p) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_sizes(fn, p->rows, p->n_in, p->n_out, p->dtype));
  if (p->act < VB_ACT_NONE || p->act > VB_ACT_SILU) return fail(VB_EINVAL, "%s: unknown activation %d", fn, p->act);
  if (p->round_g != 0 && p->round_g != 1) return fail(VB_EINVAL, "%s: round_g must be 0 or 1 (got %d)", fn, p->round_g);
  const bool some = p->rows > 0;
  TRY(check_matrix(fn, "dy", p->dy, p->ld_dy, p->n_out, p->dtype, some));
  TRY(check_matrix(fn, "x", p->x, p->ld_x, p->n_in, p->dtype, some && p->dweight));
  TRY(check_matrix(fn, "weight", p->weight, p->ld_w, p->n_in, p->dtype, some && p->dx));
  TRY(check_matrix(fn, "saved", p->saved, p->ld_saved, p->n_out, p->dtype, some && p->act != VB_ACT_NONE));
  TRY(check_matrix(fn, "dx", p->dx, p->ld_dx, p->n_in, p->dtype, false));
  TRY(check_matrix(fn, "dweight", p->dweight, p->ld_dw, p->n_in, p->dtype, false));
  TRY(check_matrix(fn, "dbias", p->dbias, p->n_out, p->n_out, p->dtype, false));
  TRY(check_matrix(fn, "dresidual", p->dresidual, p->ld_dres, p->n_out, p->dtype, false));
  // without rows dx and dresidual are empty, and may be NULL for that
  if (some && !p->dx && !p->dweight && !p->dbias && !p->dresidual) return fail(VB_EINVAL, "%s: nothing to compute", fn);
  if (p->dresidual == p->dy && p->dy && p->ld_dres != p->ld_dy)
    return fail(VB_ESHAPE, "%s: dresidual over dy needs the same leading dimension", fn);
  const hipStream_t st = (hipStream_t)stream;
  const long long es = (long long)elem_size(p->dtype);
  const BackwardCall call = backward_call(*p);
  BackwardPlan f = plan_backward(call);
  if (some) TRY(check_ws(fn, ws, ws_bytes, f.total));
  const void* saved = p->act == VB_ACT_NONE ? nullptr : p->saved;
  const Named memory[] = {matrix("dresidual", p->dresidual, p->rows, p->n_out, p->ld_dres, p->dtype, true),
                          matrix("dx", p->dx, p->rows, p->n_in, p->ld_dx, p->dtype, true),
                          matrix("dweight", p->dweight, p->n_out, p->n_in, p->ld_dw, p->dtype, true),
                          matrix("dbias", p->dbias, 1, p->n_out, p->n_out, p->dtype, true),
                          block("the workspace", ws, (int64_t)f.total, true),
                          matrix("dy", p->dy, p->rows, p->n_out, p->ld_dy, p->dtype, false),
                          matrix("x", p->dweight ? p->x : nullptr, p->rows, p->n_in, p->ld_x, p->dtype, false),
                          matrix("weight", p->dx ? p->weight : nullptr, p->n_out, p->n_in, p->ld_w, p->dtype, false),
                          matrix("saved", saved, p->rows, p->n_out, p->ld_saved, p->dtype, false)};
  TRY(check_overlaps(fn, memory, 0, 5));
  if (!some) {
    if (p->dweight) HIPCHK(launch_fill_zero(p->dweight, p->n_out, p->n_in * es, p->ld_dw * es, st));
    if (p->dbias) HIPCHK(launch_fill_zero(p->dbias, 1, p->n_out * es, p->n_out * es, st));
    return VB_OK;
  }
  const PackJobs jobs = backward_copies(call, f, ws);
  ColumnSums sums{};
  if (f.g.used || p->dbias || p->dresidual) {
    ActGrad g{};
    g.dy = p->dy, g.ld_dy = p->ld_dy;
    g.saved = saved, g.ld_saved = p->ld_saved;
    g.g = f.g.in(ws), g.g_low = f.g_low.in(ws), g.ld_g = (long long)chunked_row(p->n_out, p->dtype) / es;
    g.dres = p->dresidual, g.ld_dres = p->ld_dres;
    g.dbias = p->dbias, g.partial = (float*)f.sums.in(ws);
    g.rows = p->rows, g.n = p->n_out, g.act = p->act;
    HIPCHK(launch_act_grad(g, jobs, p->dtype, sums, st));
  } else {
    HIPCHK(launch_pack(jobs, p->dtype, st));
  }
  return run_backward(call, f, sums, ws, st);
}

extern "C" vb_status vb_cross_entropy_workspace(int64_t rows, int32_t classes, int32_t dtype, size_t* bytes) {
  if (!bytes) return fail(VB_EINVAL, "vb_cross_entropy_workspace: bytes is NULL");
  TRY(check_sizes("vb_cross_entropy_workspace", rows, classes, classes, dtype, MAX_CLASSES));
  *bytes = align_up(16 + (size_t)rows * 4);
  return VB_OK;
}

extern "C" vb_status vb_cross_entropy(const vb_cross_entropy_args* p, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "vb_cross_entropy";
  if (!p) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_sizes(fn, p->rows, p->classes, p->classes, p->dtype, MAX_CLASSES));
  const bool some = p->rows > 0;
  TRY(check_matrix(fn, "logits", p->logits, p->ld, p->classes, p->dtype, some));
  TRY(check_matrix(fn, "dlogits", p->dlogits, p->ld_d, p->classes, p->dtype, false));
  if (some && !p->labels) return fail(VB_EINVAL, "%s: labels is NULL", fn);
  if ((uintptr_t)p->labels & 7) return fail(VB_EINVAL, "%s: labels is not aligned to its elements", fn);
  if (((uintptr_t)p->loss & 3) || ((uintptr_t)p->row_loss & 3)) return fail(VB_EINVAL, "%s: loss or row_loss is not aligned to its elements", fn);
  if (!(p->label_smoothing >= 0.f && p->label_smoothing <= 1.f))
    return fail(VB_EINVAL, "%s: label_smoothing must be in [0, 1] (got %g)", fn, p->label_smoothing);
  if (!p->loss && !p->row_loss && !p->dlogits) return fail(VB_EINVAL, "%s: nothing to compute", fn);
  if (p->dlogits && p->dlogits == p->logits && p->ld_d != p->ld)
    return fail(VB_ESHAPE, "%s: dlogits over logits needs the same leading dimension", fn);
  size_t need = 0;
  TRY(vb_cross_entropy_workspace(p->rows, p->classes, p->dtype, &need));
  TRY(check_ws(fn, ws, ws_bytes, need));
  const Named memory[] = {matrix("dlogits", p->dlogits, p->rows, p->classes, p->ld_d, p->dtype, true),
                          block("loss", p->loss, 4, true), block("row_loss", p->row_loss, p->rows * 4, true),
                          block("the workspace", ws, (int64_t)need, true),
                          matrix("logits", p->logits, p->rows, p->classes, p->ld, p->dtype, false),
                          block("labels", p->labels, p->rows * 8, false)};
  TRY(check_overlaps(fn, memory, 0, 4));
  HIPCHK(launch_cross_entropy(*p, ws, (hipStream_t)stream));
  return VB_OK;
}

namespace {

// Chunks of all tensors, or -1 for a bad size or too many; their size.
long long clip_chunks(int32_t n, const int64_t* sizes, int& chunk) {
  for (int c : {CLIP_FEW_CHUNK, CLIP_CHUNK}) {
    long long count = 0;
    for (int32_t i = 0; i < n; ++i) {
      if (sizes[i] < 0 || sizes[i] > (INT64_C(1) << 44)) return -1;
      count += (sizes[i] + c - 1) / c;
      if (count > CLIP_MAX_CHUNKS && c == CLIP_CHUNK) return -1;
    }
    chunk = c;
    if (c == CLIP_CHUNK || count <= CLIP_FEW) return count;
  }
  return -1;
}

struct ClipCall {
  int32_t n_tensors;
  const void* const* grads;
  void* const* out;
  const int64_t* sizes;
  const int32_t* dtypes;
  float max_norm;
  float* norm;
  void* ws;
  hipStream_t st;
};

// As check_overlaps, of any number of tensors: their spans in the order of memory.  An
// output that is its own gradient is one span.
vb_status check_clip_overlaps(const char* fn, const ClipCall& c, size_t ws_bytes) {
  struct Item {
    uintptr_t at, end;
    bool written;
  };
  constexpr int FEW = 64;
  Item few[2 * FEW + 2], *item = few;
  if (c.n_tensors > FEW && !(item = new (std::nothrow) Item[2 * (size_t)c.n_tensors + 2]))
    return fail(VB_ENOMEM, "%s: no host memory for %d tensors", fn, c.n_tensors);
  size_t n = 0;
  auto add = [&](const void* p, size_t bytes, bool written) {
    if (bytes) item[n++] = {(uintptr_t)p, (uintptr_t)p + bytes, written};
  };
  add(c.norm, 4, true);
  add(c.ws, ws_bytes, true);
  for (int32_t i = 0; i < c.n_tensors; ++i) {
    const size_t bytes = (size_t)c.sizes[i] * elem_size(c.dtypes[i]);
    const bool apart = c.out && c.out[i] != c.grads[i];
    add(c.grads[i], bytes, !apart);
    if (apart) add(c.out[i], bytes, true);
  }
  std::sort(item, item + n, [](const Item& a, const Item& b) { return a.at < b.at; });
  uintptr_t end = 0, written_end = 0;  // of what starts before
  bool clash = false;
  for (size_t i = 0; i < n; ++i) {
    clash |= item[i].at < (item[i].written ? end : written_end);
    end = std::max(end, item[i].end);
    if (item[i].written) written_end = std::max(written_end, item[i].end);
  }
  if (item != few) delete[] item;
  return clash ? fail(VB_EINVAL, "%s: a tensor that is written overlaps another one", fn) : VB_OK;
}

template <int N>
vb_status run_clip(const ClipCall& c) {
  // the next tensors, from number i on, in chunks of `chunk`
  int32_t i = 0;
  auto fill = [&](ClipTable<N>& t, int chunk) {
    t.count = 0;
    t.chunk = chunk;
    t.first[0] = 0;
    for (; i < c.n_tensors && t.count < N; ++i) {
      if (c.sizes[i] == 0) continue;
      const int k = t.count++;
      t.grad[k] = c.grads[i];
      t.out[k] = c.out ? c.out[i] : (void*)c.grads[i];
      t.n[k] = c.sizes[i];
      t.dtype[k] = (unsigned char)c.dtypes[i];
      t.first[k + 1] = t.first[k] + (unsigned)((c.sizes[i] + chunk - 1) / chunk);
    }
    return t.count > 0;
  };
  ClipTable<N> t;
  // one workgroup for few numbers, also for none at all, when the norm is written all the same
  long long total = 0;
  int32_t filled = 0;
  for (int32_t k = 0; k < c.n_tensors; ++k) total += c.sizes[k], filled += c.sizes[k] > 0;
  if (total <= CLIP_SMALL && filled <= N) {
    fill(t, CLIP_SMALL_CHUNK);
    HIPCHK(launch_clip_small(t, c.max_norm, c.norm, c.st));
    return VB_OK;
  }
  int chunk = 0;
  const long long chunks = clip_chunks(c.n_tensors, c.sizes, chunk);
  float* scale = (float*)c.ws;
  double* partial = (double*)((char*)c.ws + 16);
  long long at = 0;
  while (fill(t, chunk)) {
    HIPCHK(launch_clip_partial(t, partial + at, c.st));
    at += t.first[t.count];
  }
  const bool few = chunks <= CLIP_FEW;
  if (!few) HIPCHK(launch_clip_norm(partial, at, c.max_norm, c.norm, scale, c.st));
  i = 0;
  for (float* write = c.norm; fill(t, chunk); write = nullptr)
    HIPCHK(launch_clip_scale(t, scale, partial, few ? (int)chunks : 0, c.max_norm, write, c.st));
  return VB_OK;
}

}  // namespace

extern "C" vb_status vb_clip_grad_norm_workspace(int32_t n_tensors, const int64_t* sizes, size_t* bytes) {
  const char* fn = "vb_clip_grad_norm_workspace";
  if (!bytes) return fail(VB_EINVAL, "%s: bytes is NULL", fn);
  if (n_tensors < 0 || (n_tensors > 0 && !sizes)) return fail(VB_EINVAL, "%s: bad tensor list", fn);
  int chunk = 0;
  const long long chunks = clip_chunks(n_tensors, sizes, chunk);
  if (chunks < 0) return fail(VB_EINVAL, "%s: a size is negative or the total too large", fn);
  *bytes = align_up(16 + (size_t)chunks * 8);
  return VB_OK;
}

extern "C" vb_status vb_clip_grad_norm(int32_t n_tensors, const void* const* grads, void* const* out,
                                       const int64_t* sizes, const int32_t* dtypes, float max_norm, float* norm,
                                       void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "vb_clip_grad_norm";
  if (n_tensors < 0 || (n_tensors > 0 && (!grads || !sizes || !dtypes))) return fail(VB_EINVAL, "%s: bad tensor list", fn);
  if (!norm || ((uintptr_t)norm & 3)) return fail(VB_EINVAL, "%s: norm is NULL or misaligned", fn);
  if (!(max_norm >= 0.f)) return fail(VB_EINVAL, "%s: max_norm must be >= 0 (got %g)", fn, max_norm);
  size_t need = 0;
  TRY(vb_clip_grad_norm_workspace(n_tensors, sizes, &need));
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (dtypes[i] < VB_F32 || dtypes[i] > VB_F16) return fail(VB_EINVAL, "%s: unknown dtype %d of tensor %d", fn, dtypes[i], i);
    if (sizes[i] == 0) continue;
    const uintptr_t es = elem_size(dtypes[i]);
    if (!grads[i] || (uintptr_t)grads[i] % es || (out && (!out[i] || (uintptr_t)out[i] % es)))
      return fail(VB_EINVAL, "%s: pointer of tensor %d is NULL or misaligned", fn, i);
  }
  TRY(check_ws(fn, ws, ws_bytes, need));
  const ClipCall c{n_tensors, grads, out, sizes, dtypes, max_norm, norm, ws, (hipStream_t)stream};
  TRY(check_clip_overlaps(fn, c, need));
  return n_tensors <= CLIP_FEW_TENSORS ? run_clip<CLIP_FEW_TENSORS>(c) : run_clip<CLIP_TENSORS>(c);
}
