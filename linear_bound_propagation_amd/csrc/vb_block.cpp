// C ABI of the gated linear layer, layer norm and dropout (include/vb_train.h): argument
// checks and the sequence of launches.  Nothing here throws.
#include <cmath>

#include "vb_train.h"
#include "vb_train_host.h"

using namespace vb;

namespace {

// W has 2 n_out rows, so n_out is half of a layer's widest.
vb_status check_gated(const char* fn, int64_t rows, int32_t n_in, int32_t n_out, int32_t dtype) {
  TRY(check_sizes(fn, rows, n_in, n_out, dtype));
  if (n_out > MAX_WIDTH / 2) return fail(VB_EUNSUPPORTED, "%s: n_out above %d is not supported (got %d)", fn, MAX_WIDTH / 2, n_out);
  return VB_OK;
}

vb_status check_act(const char* fn, int32_t act) {
  return act < VB_ACT_NONE || act > VB_ACT_SILU ? fail(VB_EINVAL, "%s: unknown activation %d", fn, act) : VB_OK;
}

// The product, and copies of operands whose rows a large product cannot read.
struct GatedPlan {
  Product d{};
  Part x, w, partial;
  size_t total = 0;
};

GatedPlan plan_gated(const vb_gated_linear_fwd& p) {
  GatedPlan f;
  Product& d = f.d;
  d.a = p.x, d.lda = p.ld_x;
  d.b = p.weight, d.ldb = p.ld_w;
  d.M = p.rows, d.N = p.n_out, d.K = p.n_in, d.passes = 1, d.gated = true;
  d.bias = p.bias, d.act = p.act;
  d.out = p.y, d.ld_out = p.ld_y, d.pre = p.pre, d.ld_pre = p.ld_pre;
  if (p.rows == 0 || product_is_narrow(d, p.dtype)) return f;
  d.tiled = true;
  const size_t row = chunked_row(p.n_in, p.dtype);
  if (!is_chunked(p.x, p.ld_x, p.n_in, p.dtype)) f.x.take(f.total, p.rows * row);
  if (!is_chunked(p.weight, p.ld_w, p.n_in, p.dtype)) f.w.take(f.total, 2 * (size_t)p.n_out * row);
  f.partial.take(f.total, product_bytes(d, p.dtype));
  return f;
}

BackwardCall backward_call(const vb_gated_linear_bwd& p) {
  BackwardCall c{};
  c.rows = p.rows, c.n_in = p.n_in, c.n_g = 2 * p.n_out, c.dtype = p.dtype;
  c.make_g = true;
  c.two = p.dtype != VB_F32 && !p.round_g;
  c.x = p.x, c.ld_x = p.ld_x, c.weight = p.weight, c.ld_w = p.ld_w;
  c.dx = p.dx, c.ld_dx = p.ld_dx, c.dweight = p.dweight, c.ld_dw = p.ld_dw;
  if (p.dbias && p.rows > 0) c.sums_bytes = gate_grad_bytes(p.rows, p.n_out, p.dtype);
  return c;
}

// Zeros for the gradients of parameters that no row reaches.
vb_status fill_zero(void* p, int64_t rows, int64_t n, int64_t ld, int dtype, hipStream_t st) {
  const long long es = (long long)elem_size(dtype);
  if (p) HIPCHK(launch_fill_zero(p, rows, n * es, ld * es, st));
  return VB_OK;
}

}  // namespace

extern "C" vb_status vb_gated_linear_forward_workspace(const vb_gated_linear_fwd* p, size_t* bytes) {
  const char* fn = "vb_gated_linear_forward_workspace";
  if (!p || !bytes) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_gated(fn, p->rows, p->n_in, p->n_out, p->dtype));
  *bytes = plan_gated(*p).total;
  return VB_OK;
}

extern "C" vb_status vb_gated_linear_backward_workspace(const vb_gated_linear_bwd* p, size_t* bytes) {
  const char* fn = "vb_gated_linear_backward_workspace";
  if (!p || !bytes) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_gated(fn, p->rows, p->n_in, p->n_out, p->dtype));
  *bytes = plan_backward(backward_call(*p)).total;
  return VB_OK;
}

extern "C" vb_status vb_gated_linear_forward(const vb_gated_linear_fwd* p, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "vb_gated_linear_forward";
  if (!p) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_gated(fn, p->rows, p->n_in, p->n_out, p->dtype));
  TRY(check_act(fn, p->act));
  if (p->rows == 0) return VB_OK;
  const int64_t n2 = 2 * (int64_t)p->n_out;
  TRY(check_matrix(fn, "x", p->x, p->ld_x, p->n_in, p->dtype, true));
  TRY(check_matrix(fn, "weight", p->weight, p->ld_w, p->n_in, p->dtype, true));
  TRY(check_matrix(fn, "bias", p->bias, n2, n2, p->dtype, false));
  TRY(check_matrix(fn, "y", p->y, p->ld_y, p->n_out, p->dtype, true));
  TRY(check_matrix(fn, "pre", p->pre, p->ld_pre, n2, p->dtype, false));
  GatedPlan f = plan_gated(*p);
  TRY(check_ws(fn, ws, ws_bytes, f.total));
  const Named memory[] = {matrix("y", p->y, p->rows, p->n_out, p->ld_y, p->dtype, true),
                          matrix("pre", p->pre, p->rows, n2, p->ld_pre, p->dtype, true),
                          block("the workspace", ws, (int64_t)f.total, true),
                          matrix("x", p->x, p->rows, p->n_in, p->ld_x, p->dtype, false),
                          matrix("weight", p->weight, n2, p->n_in, p->ld_w, p->dtype, false),
                          matrix("bias", p->bias, 1, n2, n2, p->dtype, false)};
  TRY(check_overlaps(fn, memory));
  const hipStream_t st = (hipStream_t)stream;
  const long long ld = (long long)(chunked_row(p->n_in, p->dtype) / elem_size(p->dtype));
  HIPCHK(launch_pack({{{p->x, p->ld_x, p->rows, p->n_in, f.x.in(ws)}, {p->weight, p->ld_w, n2, p->n_in, f.w.in(ws)}}},
                     p->dtype, st));
  if (f.x.used) f.d.a = f.x.in(ws), f.d.lda = ld;
  if (f.w.used) f.d.b = f.w.in(ws), f.d.ldb = ld;
  f.d.partial = (float*)f.partial.in(ws);
  HIPCHK(launch_product(f.d, p->dtype, st));
  return VB_OK;
}

extern "C" vb_status vb_gated_linear_backward(const vb_gated_linear_bwd* p, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "vb_gated_linear_backward";
  if (!p) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_gated(fn, p->rows, p->n_in, p->n_out, p->dtype));
  TRY(check_act(fn, p->act));
  if (p->round_g != 0 && p->round_g != 1) return fail(VB_EINVAL, "%s: round_g must be 0 or 1 (got %d)", fn, p->round_g);
  const bool some = p->rows > 0;
  const int64_t n2 = 2 * (int64_t)p->n_out;
  TRY(check_matrix(fn, "dy", p->dy, p->ld_dy, p->n_out, p->dtype, some));
  TRY(check_matrix(fn, "x", p->x, p->ld_x, p->n_in, p->dtype, some && p->dweight));
  TRY(check_matrix(fn, "weight", p->weight, p->ld_w, p->n_in, p->dtype, some && p->dx));
  TRY(check_matrix(fn, "pre", p->pre, p->ld_pre, n2, p->dtype, some));
  TRY(check_matrix(fn, "dx", p->dx, p->ld_dx, p->n_in, p->dtype, false));
  TRY(check_matrix(fn, "dweight", p->dweight, p->ld_dw, p->n_in, p->dtype, false));
  TRY(check_matrix(fn, "dbias", p->dbias, n2, n2, p->dtype, false));
  // without rows dx is empty, and may be NULL for that
  if (some && !p->dx && !p->dweight && !p->dbias) return fail(VB_EINVAL, "%s: nothing to compute", fn);
  const BackwardCall call = backward_call(*p);
  BackwardPlan f = plan_backward(call);
  TRY(check_ws(fn, ws, ws_bytes, f.total));
  const Named memory[] = {matrix("dx", p->dx, p->rows, p->n_in, p->ld_dx, p->dtype, true),
                          matrix("dweight", p->dweight, n2, p->n_in, p->ld_dw, p->dtype, true),
                          matrix("dbias", p->dbias, 1, n2, n2, p->dtype, true),
                          block("the workspace", ws, (int64_t)f.total, true),
                          matrix("dy", p->dy, p->rows, p->n_out, p->ld_dy, p->dtype, false),
                          matrix("x", p->dweight ? p->x : nullptr, p->rows, p->n_in, p->ld_x, p->dtype, false),
                          matrix("weight", p->dx ? p->weight : nullptr, n2, p->n_in, p->ld_w, p->dtype, false),
                          matrix("pre", p->pre, p->rows, n2, p->ld_pre, p->dtype, false)};
  TRY(check_overlaps(fn, memory));
  const hipStream_t st = (hipStream_t)stream;
  if (!some) {
    TRY(fill_zero(p->dweight, n2, p->n_in, p->ld_dw, p->dtype, st));
    return fill_zero(p->dbias, 1, n2, n2, p->dtype, st);
  }
  GateGrad g{};
  g.dy = p->dy, g.ld_dy = p->ld_dy, g.pre = p->pre, g.ld_pre = p->ld_pre;
  g.g = f.g.in(ws), g.g_low = f.g_low.in(ws), g.ld_g = (long long)(chunked_row(n2, p->dtype) / elem_size(p->dtype));
  g.dbias = p->dbias, g.partial = (float*)f.sums.in(ws);
  g.rows = p->rows, g.n = p->n_out, g.act = p->act;
  ColumnSums sums{};
  HIPCHK(launch_gate_grad(g, backward_copies(call, f, ws), p->dtype, sums, st));
  return run_backward(call, f, sums, ws, st);
}

extern "C" vb_status vb_layer_norm_forward(const vb_layer_norm_fwd* p, void* stream) {
  const char* fn = "vb_layer_norm_forward";
  if (!p) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_sizes(fn, p->rows, p->n, p->n, p->dtype));
  if (!(p->eps >= 0.f) || std::isinf(p->eps)) return fail(VB_EINVAL, "%s: eps must be finite and >= 0 (got %g)", fn, p->eps);
  if (p->rows == 0) return VB_OK;
  TRY(check_matrix(fn, "x", p->x, p->ld_x, p->n, p->dtype, true));
  TRY(check_matrix(fn, "y", p->y, p->ld_y, p->n, p->dtype, true));
  TRY(check_matrix(fn, "weight", p->weight, p->n, p->n, p->dtype, false));
  TRY(check_matrix(fn, "bias", p->bias, p->n, p->n, p->dtype, false));
  TRY(check_matrix(fn, "mean", p->mean, p->rows, p->rows, VB_F32, false, MAX_ROWS));
  TRY(check_matrix(fn, "rstd", p->rstd, p->rows, p->rows, VB_F32, false, MAX_ROWS));
  if (p->y == p->x && p->ld_y != p->ld_x) return fail(VB_ESHAPE, "%s: y over x needs the same leading dimension", fn);
  const Named memory[] = {matrix("y", p->y, p->rows, p->n, p->ld_y, p->dtype, true),
                          block("mean", p->mean, p->rows * 4, true), block("rstd", p->rstd, p->rows * 4, true),
                          matrix("x", p->x, p->rows, p->n, p->ld_x, p->dtype, false),
                          matrix("weight", p->weight, 1, p->n, p->n, p->dtype, false),
                          matrix("bias", p->bias, 1, p->n, p->n, p->dtype, false)};
  TRY(check_overlaps(fn, memory, 0, 3));
  HIPCHK(launch_layer_norm(*p, (hipStream_t)stream));
  return VB_OK;
}

extern "C" vb_status vb_layer_norm_backward_workspace(int64_t rows, int32_t n, int32_t dtype, size_t* bytes) {
  const char* fn = "vb_layer_norm_backward_workspace";
  if (!bytes) return fail(VB_EINVAL, "%s: bytes is NULL", fn);
  TRY(check_sizes(fn, rows, n, n, dtype));
  *bytes = rows ? align_up(norm_grad_bytes(rows, n, dtype)) : 0;
  return VB_OK;
}

extern "C" vb_status vb_layer_norm_backward(const vb_layer_norm_bwd* p, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "vb_layer_norm_backward";
  if (!p) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_sizes(fn, p->rows, p->n, p->n, p->dtype));
  const bool some = p->rows > 0;
  TRY(check_matrix(fn, "dy", p->dy, p->ld_dy, p->n, p->dtype, some));
  TRY(check_matrix(fn, "x", p->x, p->ld_x, p->n, p->dtype, some));
  TRY(check_matrix(fn, "mean", p->mean, p->rows, p->rows, VB_F32, some, MAX_ROWS));
  TRY(check_matrix(fn, "rstd", p->rstd, p->rows, p->rows, VB_F32, some, MAX_ROWS));
  TRY(check_matrix(fn, "weight", p->weight, p->n, p->n, p->dtype, false));
  TRY(check_matrix(fn, "dresidual", p->dresidual, p->ld_dres, p->n, p->dtype, false));
  TRY(check_matrix(fn, "dx", p->dx, p->ld_dx, p->n, p->dtype, false));
  TRY(check_matrix(fn, "dweight", p->dweight, p->n, p->n, p->dtype, false));
  TRY(check_matrix(fn, "dbias", p->dbias, p->n, p->n, p->dtype, false));
  // without rows dx is empty, and may be NULL for that
  if (some && !p->dx && !p->dweight && !p->dbias) return fail(VB_EINVAL, "%s: nothing to compute", fn);
  if (p->dx && p->dx == p->dy && p->ld_dx != p->ld_dy)
    return fail(VB_ESHAPE, "%s: dx over dy needs the same leading dimension", fn);
  if (p->dx && p->dx == p->dresidual && p->ld_dx != p->ld_dres)
    return fail(VB_ESHAPE, "%s: dx over dresidual needs the same leading dimension", fn);
  size_t need = 0;
  if (p->dweight || p->dbias) TRY(vb_layer_norm_backward_workspace(p->rows, p->n, p->dtype, &need));
  TRY(check_ws(fn, ws, ws_bytes, need));
  const Named memory[] = {matrix("dx", p->dx, p->rows, p->n, p->ld_dx, p->dtype, true),
                          matrix("dweight", p->dweight, 1, p->n, p->n, p->dtype, true),
                          matrix("dbias", p->dbias, 1, p->n, p->n, p->dtype, true),
                          block("the workspace", ws, (int64_t)need, true),
                          matrix("dy", p->dy, p->rows, p->n, p->ld_dy, p->dtype, false),
                          matrix("dresidual", p->dx ? p->dresidual : nullptr, p->rows, p->n, p->ld_dres, p->dtype, false),
                          matrix("x", p->x, p->rows, p->n, p->ld_x, p->dtype, false),
                          block("mean", p->mean, p->rows * 4, false),
                          block("rstd", p->rstd, p->rows * 4, false),
                          matrix("weight", p->dx ? p->weight : nullptr, 1, p->n, p->n, p->dtype, false)};
  TRY(check_overlaps(fn, memory, 0, 4, 5));
  const hipStream_t st = (hipStream_t)stream;
  if (!some) {
    TRY(fill_zero(p->dweight, 1, p->n, p->n, p->dtype, st));
    return fill_zero(p->dbias, 1, p->n, p->n, p->dtype, st);
  }
  HIPCHK(launch_layer_norm_grad(*p, (float*)ws, st));
  return VB_OK;
}

extern "C" vb_status vb_dropout(const vb_dropout_args* p, void* stream) {
  const char* fn = "vb_dropout";
  if (!p) return fail(VB_EINVAL, "%s: NULL argument", fn);
  TRY(check_sizes(fn, p->rows, p->n, p->n, p->dtype, MAX_CLASSES));
  if (!(p->p >= 0. && p->p <= 1.)) return fail(VB_EINVAL, "%s: p must be in [0, 1] (got %g)", fn, p->p);
  if (p->rows == 0) return VB_OK;
  TRY(check_matrix(fn, "x", p->x, p->ld_x, p->n, p->dtype, true));
  TRY(check_matrix(fn, "residual", p->residual, p->ld_res, p->n, p->dtype, false));
  TRY(check_matrix(fn, "y", p->y, p->ld_y, p->n, p->dtype, true));
  if ((uintptr_t)p->step & 7) return fail(VB_EINVAL, "%s: step is not aligned to its elements", fn);
  if (p->y == p->x && p->ld_y != p->ld_x) return fail(VB_ESHAPE, "%s: y over x needs the same leading dimension", fn);
  if (p->y == p->residual && p->ld_y != p->ld_res)
    return fail(VB_ESHAPE, "%s: y over residual needs the same leading dimension", fn);
  const Named memory[] = {matrix("y", p->y, p->rows, p->n, p->ld_y, p->dtype, true),
                          matrix("x", p->x, p->rows, p->n, p->ld_x, p->dtype, false),
                          matrix("residual", p->residual, p->rows, p->n, p->ld_res, p->dtype, false),
                          block("step", p->step, 8, false)};
  TRY(check_overlaps(fn, memory, 0, 1, 2));
  HIPCHK(launch_dropout(*p, (hipStream_t)stream));
  return VB_OK;
}
