/* vb_train.h -- C ABI of the training and evaluation operators in libvbprop.so.
 *
 * The networks whose bounds vb.h computes are evaluated and trained with these
 * calls: the fused linear layer and its backward pass, the softmax cross
 * entropy with its gradient, and the clipping of gradients to a global norm.
 *
 * Conventions (those of vb.h, where they apply):
 *  - Tensor pointers are DEVICE pointers owned by the caller; nothing is kept
 *    after a call returns and no device memory is allocated.  Scratch comes
 *    from the caller's workspace `ws` (16-byte aligned), whose size the
 *    vb_*_workspace calls give; its contents before and after a call mean
 *    nothing.  Calls that may overlap need a workspace each.
 *  - Every call validates its arguments on the host first.  On an error nothing
 *    is enqueued and a negative status is returned; vb_last_error() describes
 *    it.  Otherwise the work is enqueued on `stream` and the call returns
 *    without synchronising.  The calls may be captured into a HIP graph.
 *  - Results are deterministic: identical inputs give bitwise-identical outputs
 *    (all sums run in a fixed order, no float atomics).
 *  - Matrices are row-major with a leading dimension (elements between rows) of
 *    at least the row length.  Data of a call has one type (dtype); sums,
 *    statistics and everything between input and output are float32 or wider,
 *    and an output is rounded once (to nearest even), except where a call says
 *    otherwise.  Any element alignment is accepted; rows that start on 16-byte
 *    boundaries are faster.
 *  - Infinities and NaN follow the formulas.
 *  - What a call writes shares no memory with its other arguments, except where the
 *    call names an output that may be an input itself.  Overlaps are refused; rows
 *    of one matrix between those of another (column ranges of one buffer) are none.
 */
#ifndef VB_TRAIN_H
#define VB_TRAIN_H

#include "vb.h"

#ifdef __cplusplus
extern "C" {
#endif

#define VB_F32  0
#define VB_BF16 1
#define VB_F16  2

#define VB_ACT_NONE 0
#define VB_ACT_RELU 1   /* max(v, 0)                        */
#define VB_ACT_GELU 2   /* v Phi(v), Phi the normal CDF     */
#define VB_ACT_SILU 3   /* v / (1 + exp(-v))                */

/* The fused linear layer: pre = x W^T + bias + residual, y = act(pre).
 * With a residual and a ReLU this is the last step of a residual block; with a
 * residual and no activation, of a pre-norm block. */
typedef struct {
  int64_t rows;                          /* >= 0 (0: nothing is enqueued)          */
  int32_t n_in, n_out;                   /* in [1, 2^20]                           */
  int32_t dtype, act;                    /* VB_F32 .., VB_ACT_NONE ..              */
  const void* x;        int64_t ld_x;    /* [rows][n_in]                           */
  const void* weight;   int64_t ld_w;    /* [n_out][n_in]                          */
  const void* bias;                      /* [n_out] or NULL                        */
  const void* residual; int64_t ld_res;  /* [rows][n_out] or NULL                  */
  void* y;              int64_t ld_y;    /* [rows][n_out]; may be residual itself  */
                                         /* (the same pointer and ld)              */
  void* pre;            int64_t ld_pre;  /* [rows][n_out] or NULL: pre, rounded to */
                                         /* dtype, for the backward pass of        */
                                         /* VB_ACT_GELU / VB_ACT_SILU              */
} vb_linear_fwd;

/* Its backward pass for the gradient dy of y, with g = dy * act'(pre):
 *   dx = g W, dweight = g^T x, dbias = column sums of g, dresidual = g.
 * saved: NULL for VB_ACT_NONE; y for VB_ACT_RELU (act' = 1 where y > 0, 0
 * elsewhere: where saved is not > 0, g is 0 whatever dy holds); pre for GELU
 * and SILU.  dx, dweight, dbias and dresidual may each be NULL, with rows > 0 not
 * all of them.  With rows = 0 dweight and dbias are set to zero.  dresidual may be dy itself (same pointer
 * and ld).
 * The matrix cores take operands of dtype.  With GELU and SILU in a 16-bit type g
 * is no number of that type: it enters both products as the sum of two (relative
 * error 2^-16 in bfloat16, 2^-22 in float16), which multiplies twice, or, with
 * round_g, rounded to one, which takes half the time and adds an error as large
 * as the rounding of the gradients themselves.  dbias sums the unrounded g. */
typedef struct {
  int64_t rows;
  int32_t n_in, n_out;
  int32_t dtype, act;
  const void* dy;       int64_t ld_dy;   /* [rows][n_out]           */
  const void* x;        int64_t ld_x;    /* [rows][n_in]            */
  const void* weight;   int64_t ld_w;    /* [n_out][n_in]           */
  const void* saved;    int64_t ld_saved;/* [rows][n_out] or NULL   */
  void* dx;             int64_t ld_dx;   /* [rows][n_in] or NULL    */
  void* dweight;        int64_t ld_dw;   /* [n_out][n_in] or NULL   */
  void* dbias;                           /* [n_out] or NULL         */
  void* dresidual;      int64_t ld_dres; /* [rows][n_out] or NULL   */
  int32_t round_g;                       /* 0 or 1                  */
} vb_linear_bwd;

/* Workspace of a call with these arguments.  Of the pointers only x, weight and dy are
 * looked at, for their alignment (rows that do not start on 16-byte boundaries or are no
 * whole number of 16 bytes are copied before a large product), and whether the others
 * are NULL; nothing is read through them. */
vb_status vb_linear_forward_workspace(const vb_linear_fwd* p, size_t* bytes);
vb_status vb_linear_backward_workspace(const vb_linear_bwd* p, size_t* bytes);
vb_status vb_linear_forward(const vb_linear_fwd* p, void* ws, size_t ws_bytes, void* stream);
vb_status vb_linear_backward(const vb_linear_bwd* p, void* ws, size_t ws_bytes, void* stream);

/* Softmax cross entropy of integer labels, and its gradient in the same call.
 * Row r with label t = labels[r] (p = softmax of the row, e = label_smoothing):
 *   row_loss[r] = (1 - e) (-log p_t) + e mean_j (-log p_j)
 *   loss        = sum of row_loss / n, n the number of rows not ignored
 *   dlogits[r]  = grad_scale / n * (p - (1 - e) onehot(t) - e / classes)
 * A row with t == ignore_index has row_loss 0 and gradient 0 and does not
 * count; with every row ignored (or rows = 0) loss is 0.  A label outside
 * [0, classes) that is not ignore_index makes its row's loss and gradient NaN
 * (and counts), so that it cannot pass unseen.  A logit of -inf (a masked class)
 * has p = 0: without smoothing its gradient is 0 and the row's loss does not feel
 * it; with smoothing the formula holds as it stands, with a gradient of
 * -e / classes * grad_scale / n and a row_loss of +inf.  A row with no finite
 * logit gives NaN, as the formula does. */
typedef struct {
  int64_t rows;                          /* >= 0                                   */
  int32_t classes;                       /* > 0                                    */
  int32_t dtype;                         /* of logits and dlogits                  */
  const void* logits;   int64_t ld;      /* [rows][classes]                        */
  const int64_t* labels;                 /* [rows]                                 */
  int64_t ignore_index;
  float label_smoothing;                 /* in [0, 1]                              */
  float grad_scale;
  float* loss;                           /* [1] or NULL                            */
  float* row_loss;                       /* [rows] or NULL                         */
  void* dlogits;        int64_t ld_d;    /* [rows][classes] or NULL; may be logits */
                                         /* itself (same pointer and ld)           */
} vb_cross_entropy_args;

vb_status vb_cross_entropy_workspace(int64_t rows, int32_t classes, int32_t dtype, size_t* bytes);
vb_status vb_cross_entropy(const vb_cross_entropy_args* p, void* ws, size_t ws_bytes, void* stream);

/* The global norm of n_tensors gradients, and clipping to it:
 *   norm = sqrt(sum of squares over all tensors)  (summed in float64)
 *   out_i = grads_i * (norm > max_norm ? max_norm / norm : 1)
 * A norm that is infinite or NaN leaves the values as they are (out_i =
 * grads_i): the caller sees it in `norm` and skips the step.
 *   grads, out, sizes, dtypes: host arrays [n_tensors]; out_i is grads_i itself
 *   (then nothing is written when nothing is clipped) or a tensor of the same
 *   size and type; out NULL: in place; sizes may be 0 (pointers then unused).
 *   max_norm: >= 0 (may be infinite: only the norm is wanted); norm: [1]
 *   float32 on the device. */
vb_status vb_clip_grad_norm_workspace(int32_t n_tensors, const int64_t* sizes, size_t* bytes);
vb_status vb_clip_grad_norm(int32_t n_tensors, const void* const* grads, void* const* out, const int64_t* sizes,
                            const int32_t* dtypes, float max_norm, float* norm, void* ws, size_t ws_bytes,
                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VB_TRAIN_H */
