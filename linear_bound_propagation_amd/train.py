"""Training and evaluation of the networks whose bounds the package computes: the fused
linear layer and its backward pass, dropout, the softmax cross entropy with its gradient
and the clipping of gradients to a global norm; and, for feed-forward blocks of networks
that it does not bound, the gated linear layer and layer norm with their backward passes
(include/vb_train.h).

Thin ctypes binding, like the rest of the package: every step runs in the
library's HIP kernels on the current stream; results are new tensors on it.
Matrices may have any row stride; elements of a row are contiguous.
No autograd graph is recorded: the gradients are calls of their own, and a tensor that
requires grad is refused unless torch.no_grad() says that its graph is not wanted.
"""
from __future__ import annotations

import ctypes
import struct
from array import array
from typing import List, Optional, Sequence, Tuple

import torch

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}

EXPORTS = ["vb_linear_forward_workspace", "vb_linear_backward_workspace", "vb_linear_forward",
           "vb_linear_backward", "vb_cross_entropy_workspace", "vb_cross_entropy", "vb_clip_grad_norm_workspace", "vb_clip_grad_norm",
           "vb_gated_linear_forward_workspace", "vb_gated_linear_backward_workspace", "vb_gated_linear_forward",
           "vb_gated_linear_backward", "vb_layer_norm_backward_workspace", "vb_layer_norm_forward",
           "vb_layer_norm_backward", "vb_dropout"]

_P, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_u64, _f64 = ctypes.c_uint64, ctypes.c_double


class vb_linear_fwd(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n_in", _i32), ("n_out", _i32), ("dtype", _i32), ("act", _i32),
                ("x", _P), ("ld_x", _i64), ("weight", _P), ("ld_w", _i64), ("bias", _P),
                ("residual", _P), ("ld_res", _i64), ("y", _P), ("ld_y", _i64), ("pre", _P), ("ld_pre", _i64)]


class vb_linear_bwd(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n_in", _i32), ("n_out", _i32), ("dtype", _i32), ("act", _i32),
                ("dy", _P), ("ld_dy", _i64), ("x", _P), ("ld_x", _i64), ("weight", _P), ("ld_w", _i64),
                ("saved", _P), ("ld_saved", _i64), ("dx", _P), ("ld_dx", _i64), ("dweight", _P), ("ld_dw", _i64),
                ("dbias", _P), ("dresidual", _P), ("ld_dres", _i64), ("round_g", _i32)]


class vb_cross_entropy_args(ctypes.Structure):
    _fields_ = [("rows", _i64), ("classes", _i32), ("dtype", _i32), ("logits", _P), ("ld", _i64), ("labels", _P),
                ("ignore_index", _i64), ("label_smoothing", _f32), ("grad_scale", _f32), ("loss", _P),
                ("row_loss", _P), ("dlogits", _P), ("ld_d", _i64)]


class vb_gated_linear_fwd(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n_in", _i32), ("n_out", _i32), ("dtype", _i32), ("act", _i32),
                ("x", _P), ("ld_x", _i64), ("weight", _P), ("ld_w", _i64), ("bias", _P),
                ("y", _P), ("ld_y", _i64), ("pre", _P), ("ld_pre", _i64)]


class vb_gated_linear_bwd(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n_in", _i32), ("n_out", _i32), ("dtype", _i32), ("act", _i32),
                ("dy", _P), ("ld_dy", _i64), ("x", _P), ("ld_x", _i64), ("weight", _P), ("ld_w", _i64),
                ("pre", _P), ("ld_pre", _i64), ("dx", _P), ("ld_dx", _i64), ("dweight", _P), ("ld_dw", _i64),
                ("dbias", _P), ("round_g", _i32)]


class vb_layer_norm_fwd(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n", _i32), ("dtype", _i32), ("x", _P), ("ld_x", _i64), ("weight", _P), ("bias", _P),
                ("eps", _f32), ("y", _P), ("ld_y", _i64), ("mean", _P), ("rstd", _P)]


class vb_layer_norm_bwd(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n", _i32), ("dtype", _i32), ("dy", _P), ("ld_dy", _i64), ("x", _P), ("ld_x", _i64),
                ("mean", _P), ("rstd", _P), ("weight", _P), ("dresidual", _P), ("ld_dres", _i64), ("dx", _P),
                ("ld_dx", _i64), ("dweight", _P), ("dbias", _P)]


class vb_dropout_args(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n", _i32), ("dtype", _i32), ("x", _P), ("ld_x", _i64), ("residual", _P),
                ("ld_res", _i64), ("p", _f64), ("seed", _u64), ("offset", _u64), ("step", _P), ("y", _P), ("ld_y", _i64)]


_FWD = struct.Struct("qiiiiQqQqQQqQqQq")    # vb_linear_fwd
_BWD = struct.Struct("qiiiiQqQqQqQqQqQqQQqi4x")  # vb_linear_bwd
_LOSS = struct.Struct("qiiQqQqffQQQq")      # vb_cross_entropy_args
_GATED = struct.Struct("qiiiiQqQqQQqQq")    # vb_gated_linear_fwd
_GATED_BWD = struct.Struct("qiiiiQqQqQqQqQqQqQi4x")   # vb_gated_linear_bwd
_NORM = struct.Struct("qiiQqQQf4xQqQQ")     # vb_layer_norm_fwd
_NORM_BWD = struct.Struct("qiiQqQqQQQQqQqQQ")         # vb_layer_norm_bwd
_DROP = struct.Struct("qiiQqQqdQQQQq")      # vb_dropout_args
assert tuple(s.size for s in (_FWD, _BWD, _LOSS, _GATED, _GATED_BWD, _NORM, _NORM_BWD, _DROP)) == tuple(
    ctypes.sizeof(c) for c in (vb_linear_fwd, vb_linear_bwd, vb_cross_entropy_args, vb_gated_linear_fwd,
                               vb_gated_linear_bwd, vb_layer_norm_fwd, vb_layer_norm_bwd, vb_dropout_args))

_call = None    # the declared functions, by name


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the calls of vb_train.h (argument blocks are passed by address)."""
    psz = ctypes.POINTER(_sz)
    for name, args in (("vb_linear_forward_workspace", [_P, psz]),
                       ("vb_linear_backward_workspace", [_P, psz]),
                       ("vb_linear_forward", [_P, _P, _sz, _P]),
                       ("vb_linear_backward", [_P, _P, _sz, _P]),
                       ("vb_cross_entropy_workspace", [_i64, _i32, _i32, psz]),
                       ("vb_cross_entropy", [_P, _P, _sz, _P]),
                       ("vb_clip_grad_norm_workspace", [_i32, _P, psz]),
                       ("vb_clip_grad_norm", [_i32, _P, _P, _P, _P, _f32, _P, _P, _sz, _P]),
                       ("vb_gated_linear_forward_workspace", [_P, psz]),
                       ("vb_gated_linear_backward_workspace", [_P, psz]),
                       ("vb_gated_linear_forward", [_P, _P, _sz, _P]),
                       ("vb_gated_linear_backward", [_P, _P, _sz, _P]),
                       ("vb_layer_norm_backward_workspace", [_i64, _i32, _i32, psz]),
                       ("vb_layer_norm_forward", [_P, _P]),
                       ("vb_layer_norm_backward", [_P, _P, _sz, _P]),
                       ("vb_dropout", [_P, _P])):
        fn = getattr(lib, name)
        fn.restype = _i32
        fn.argtypes = args


def _run(name: str, *args) -> None:
    """Calls a library function; its status becomes an exception."""
    global _call
    if _call is None:
        import linear_bound_propagation_amd as pkg
        lib = pkg.lib()
        _call = {n: getattr(lib, n) for n in EXPORTS}
    status = _call[name](*args)
    if status:
        import linear_bound_propagation_amd as pkg
        pkg._check(status, name)


def _size(name: str, *args) -> int:
    out = _sz(0)
    _run(name, *args, ctypes.byref(out))
    return out.value


def _stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)


def _dtype(t: torch.Tensor) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"float32, bfloat16 or float16 expected, got {t.dtype}")
    return code


def _device(t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current GPU, got {t.device}")
    return dev


def _matrix(name: str, t: torch.Tensor, rows: int, cols: int, like: torch.Tensor) -> int:
    """Leading dimension of a [rows][cols] operand (checked against `like`'s type and device)."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}][{cols}], got {tuple(t.shape)}")
    if t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"the elements of a row of {name} must be contiguous")
    return ld if rows > 1 else max(cols, ld)


def _vector(name: str, t: torch.Tensor, n: int, like: torch.Tensor) -> None:
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}], got {tuple(t.shape)}")
    if t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")


def _no_graph(*tensors: Optional[torch.Tensor]) -> None:
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("a tensor requires grad, and no autograd graph is recorded here: call under "
                             "torch.no_grad() (or with detached tensors), and the *_backward calls or cross_entropy for gradients")


def _act(act: str) -> int:
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return code


def _workspace(n: int, device) -> torch.Tensor:
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _scratch(ws: torch.Tensor, dev: int) -> Tuple[int, int]:
    """Address and bytes of a caller's workspace; the library checks its size and alignment."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous on the current GPU, got strides {ws.stride()} on {ws.device}")
    return ws.data_ptr(), ws.nbytes


def linear_workspace(x: torch.Tensor, weight: torch.Tensor, backward: bool = False) -> torch.Tensor:
    """A workspace for `linear` calls (or `linear_backward` calls, with any activation, all
    gradients and either round_g) on tensors of these sizes, strides and alignment, to keep between
    calls (rows that start off 16-byte boundaries take more than others)."""
    _device(x)
    rows, n_in = x.shape
    n_out = weight.shape[0]
    ld_x, ld_w = _matrix("x", x, rows, n_in, x), _matrix("weight", weight, n_out, n_in, x)
    head = (rows, n_in, n_out, _dtype(x))
    if backward:
        need = [_size("vb_linear_backward_workspace",
                      _BWD.pack(*head, ACTS["silu"], 0, n_out, x.data_ptr(), ld_x, weight.data_ptr(), ld_w, 0, n_out,
                                16, n_in, 16, n_in, 16, 16, n_out, round_g)) for round_g in (0, 1)]
        return _workspace(max(need), x.device)
    p = _FWD.pack(*head, 0, x.data_ptr(), ld_x, weight.data_ptr(), ld_w, 0, 0, n_out, 16, n_out, 0, n_out)
    return _workspace(_size("vb_linear_forward_workspace", p), x.device)


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
           residual: Optional[torch.Tensor] = None, act: str = "none", want_pre: bool = False,
           out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """y = act(x W^T + bias + residual) (vb_linear_forward): x [rows][n_in], weight
    [n_out][n_in], bias [n_out], residual [rows][n_out]; act one of none, relu, gelu, silu.
    With want_pre also the value before the activation, which linear_backward needs for
    gelu and silu: (y, pre).  `out` may be the residual itself."""
    dev = _device(x)
    dt = _dtype(x)
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x and weight must be matrices")
    rows, n_in = x.shape
    n_out = weight.shape[0]
    _no_graph(x, weight, bias, residual, out)
    ld_x = _matrix("x", x, rows, n_in, x)
    ld_w = _matrix("weight", weight, n_out, n_in, x)
    if bias is not None:
        _vector("bias", bias, n_out, x)
    ld_res = n_out if residual is None else _matrix("residual", residual, rows, n_out, x)
    if out is None:
        y, ld_y = x.new_empty((rows, n_out)), n_out
    else:
        y, ld_y = out, _matrix("out", out, rows, n_out, x)
    pre = x.new_empty((rows, n_out)) if want_pre else None
    p = _FWD.pack(rows, n_in, n_out, dt, _act(act), x.data_ptr(), ld_x, weight.data_ptr(), ld_w,
                  0 if bias is None else bias.data_ptr(), 0 if residual is None else residual.data_ptr(), ld_res,
                  y.data_ptr(), ld_y, 0 if pre is None else pre.data_ptr(), n_out)
    if ws is None:
        ws = _workspace(_size("vb_linear_forward_workspace", p), x.device)
    _run("vb_linear_forward", p, *_scratch(ws, dev), _stream(dev))
    return (y, pre) if want_pre else y


def linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, act: str = "none",
                    saved: Optional[torch.Tensor] = None, want_x: bool = True, want_weight: bool = True,
                    want_bias: bool = True, want_residual: bool = False, ws: Optional[torch.Tensor] = None,
                    round_g: bool = False):
    """Gradients of `linear` (vb_linear_backward) for the gradient dy of y: (dx, dweight, dbias,
    dresidual), None where not wanted.  saved: y for relu, pre for gelu and silu.  round_g: with
    gelu or silu in a 16-bit type, dx and dweight from the gradient of pre rounded to the type, in
    about half the time."""
    dev = _device(x)
    dt = _dtype(x)
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x and weight must be matrices")
    rows, n_in = x.shape
    n_out = weight.shape[0]
    code = _act(act)
    if (saved is None) != (code == 0):
        raise ValueError("saved is the forward pass's y (relu) or pre (gelu, silu), and None without an activation")
    _no_graph(dy, x, weight, saved)
    ld_dy = _matrix("dy", dy, rows, n_out, x)
    ld_x = _matrix("x", x, rows, n_in, x)
    ld_w = _matrix("weight", weight, n_out, n_in, x)
    ld_s = n_out if saved is None else _matrix("saved", saved, rows, n_out, x)
    dx = x.new_empty((rows, n_in)) if want_x else None
    dw = x.new_empty((n_out, n_in)) if want_weight else None
    db = x.new_empty((n_out,)) if want_bias else None
    dr = x.new_empty((rows, n_out)) if want_residual else None
    p = _BWD.pack(rows, n_in, n_out, dt, code, dy.data_ptr(), ld_dy, x.data_ptr(), ld_x, weight.data_ptr(), ld_w,
                  0 if saved is None else saved.data_ptr(), ld_s, 0 if dx is None else dx.data_ptr(), n_in,
                  0 if dw is None else dw.data_ptr(), n_in, 0 if db is None else db.data_ptr(),
                  0 if dr is None else dr.data_ptr(), n_out, bool(round_g))
    if ws is None:
        ws = _workspace(_size("vb_linear_backward_workspace", p), x.device)
    _run("vb_linear_backward", p, *_scratch(ws, dev), _stream(dev))
    return dx, dw, db, dr


def cross_entropy_workspace(logits: torch.Tensor) -> torch.Tensor:
    """A workspace for `cross_entropy` calls of these sizes, to keep between calls."""
    _device(logits)
    rows, classes = logits.shape
    return _workspace(_size("vb_cross_entropy_workspace", rows, classes, _dtype(logits)), logits.device)


def cross_entropy(logits: torch.Tensor, labels: torch.Tensor, ignore_index: int = -100,
                  label_smoothing: float = 0.0, grad_scale: float = 1.0, want_grad: bool = True,
                  dlogits: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Softmax cross entropy of labels [rows] (int64) and its gradient (vb_cross_entropy): (loss [1],
    row_loss [rows], dlogits [rows][classes] or None).  loss is the mean over the rows whose label
    is not ignore_index; `dlogits` may be the logits themselves."""
    dev = _device(logits)
    dt = _dtype(logits)
    if logits.dim() != 2:
        raise ValueError("logits must be a matrix")
    _no_graph(logits, dlogits)
    rows, classes = logits.shape
    ld = _matrix("logits", logits, rows, classes, logits)
    if labels.dtype is not torch.int64 or labels.shape != (rows,) or labels.get_device() != dev \
            or not labels.is_contiguous():
        raise ValueError(f"labels must be contiguous int64 [{rows}] on {logits.device}")
    ld_d = classes
    if dlogits is not None:
        ld_d = _matrix("dlogits", dlogits, rows, classes, logits)
    elif want_grad:
        dlogits = logits.new_empty((rows, classes))
    loss, row_loss = logits.new_empty(1, dtype=torch.float32), logits.new_empty(rows, dtype=torch.float32)
    if ws is None:
        ws = cross_entropy_workspace(logits)
    p = _LOSS.pack(rows, classes, dt, logits.data_ptr(), ld, labels.data_ptr(), ignore_index, label_smoothing,
                   grad_scale, loss.data_ptr(), row_loss.data_ptr(), 0 if dlogits is None else dlogits.data_ptr(), ld_d)
    _run("vb_cross_entropy", p, *_scratch(ws, dev), _stream(dev))
    return loss, row_loss, dlogits


def clip_grad_norm_workspace(grads: Sequence[torch.Tensor]) -> torch.Tensor:
    """A workspace for `clip_grad_norm` calls on tensors of these sizes, to keep between calls."""
    if len(grads):
        _device(grads[0])
    sizes = array("q", [g.numel() for g in grads])
    return _workspace(_size("vb_clip_grad_norm_workspace", len(sizes), sizes.buffer_info()[0]),
                      grads[0].device if len(grads) else "cuda")


def _tensor_list(name: str, tensors: Sequence[torch.Tensor], dev: int):
    """Types, sizes and pointers of contiguous tensors on device dev."""
    for t in tensors:
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous, on one device")
        if t.requires_grad:
            _no_graph(t)
    try:
        types = array("i", [DTYPES[t.dtype] for t in tensors])
    except KeyError:
        raise ValueError(f"{name} must be float32, bfloat16 or float16") from None
    return types, array("q", [t.numel() for t in tensors]), array("Q", [t.data_ptr() for t in tensors])


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
                   ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, List[torch.Tensor]]:
    """Global norm of the gradients, and the gradients clipped to max_norm (vb_clip_grad_norm):
    (norm [1] float32, out).  In place without `out`; a norm that is not finite clips nothing.
    Tensors are contiguous, of any mix of the three types."""
    n = len(grads)
    dev = _device(grads[0]) if n else torch.cuda.current_device()
    types, sizes, src = _tensor_list("gradients", grads, dev)
    dst = 0
    if out is not None:
        if len(out) != n:
            raise ValueError(f"{len(out)} outputs for {n} gradients")
        out_types, out_sizes, outs = _tensor_list("outputs", out, dev)
        if out_types != types or out_sizes != sizes:
            raise ValueError("outputs must have their gradients' types and numbers of elements")
        dst = outs.buffer_info()[0]
    norm = grads[0].new_empty(1, dtype=torch.float32) if n else torch.empty(1, device=torch.device("cuda", dev))
    if ws is None:
        ws = _workspace(_size("vb_clip_grad_norm_workspace", n, sizes.buffer_info()[0]), norm.device)
    _run("vb_clip_grad_norm", n, src.buffer_info()[0], dst or None, sizes.buffer_info()[0], types.buffer_info()[0],
         max_norm, norm.data_ptr(), *_scratch(ws, dev), _stream(dev))
    return norm, list(grads if out is None else out)


def _halves(weight: torch.Tensor) -> int:
    if weight.dim() != 2 or weight.shape[0] % 2:
        raise ValueError(f"weight must be a matrix of the gate's rows and as many of up's, got {tuple(weight.shape)}")
    return weight.shape[0] // 2


def gated_linear_workspace(x: torch.Tensor, weight: torch.Tensor, backward: bool = False) -> torch.Tensor:
    """A workspace for `gated_linear` calls (or `gated_linear_backward` calls, with all gradients and
    either round_g) on tensors of these sizes, strides and alignment, to keep between calls."""
    _device(x)
    n_out = _halves(weight)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    rows, n_in = x.shape
    head = (rows, n_in, n_out, _dtype(x), ACTS["silu"])
    ld_x, ld_w = _matrix("x", x, rows, n_in, x), _matrix("weight", weight, 2 * n_out, n_in, x)
    if backward:
        need = [_size("vb_gated_linear_backward_workspace",
                      _GATED_BWD.pack(*head, 0, n_out, x.data_ptr(), ld_x, weight.data_ptr(), ld_w, 0, 2 * n_out,
                                      16, n_in, 16, n_in, 16, round_g)) for round_g in (0, 1)]
        return _workspace(max(need), x.device)
    p = _GATED.pack(*head, x.data_ptr(), ld_x, weight.data_ptr(), ld_w, 0, 16, n_out, 0, 2 * n_out)
    return _workspace(_size("vb_gated_linear_forward_workspace", p), x.device)


def gated_linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "silu",
                 want_pre: bool = False, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """y = act(gate) * up with (gate | up) = x W^T + bias (vb_gated_linear_forward): x [rows][n_in],
    weight [2 n_out][n_in], the gate's rows first, bias [2 n_out]; act one of none, relu, gelu, silu.
    With want_pre also (gate | up) [rows][2 n_out], which gated_linear_backward needs: (y, pre)."""
    dev = _device(x)
    dt = _dtype(x)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    rows, n_in = x.shape
    n_out = _halves(weight)
    _no_graph(x, weight, bias, out)
    ld_x = _matrix("x", x, rows, n_in, x)
    ld_w = _matrix("weight", weight, 2 * n_out, n_in, x)
    if bias is not None:
        _vector("bias", bias, 2 * n_out, x)
    if out is None:
        y, ld_y = x.new_empty((rows, n_out)), n_out
    else:
        y, ld_y = out, _matrix("out", out, rows, n_out, x)
    pre = x.new_empty((rows, 2 * n_out)) if want_pre else None
    p = _GATED.pack(rows, n_in, n_out, dt, _act(act), x.data_ptr(), ld_x, weight.data_ptr(), ld_w,
                    0 if bias is None else bias.data_ptr(), y.data_ptr(), ld_y, 0 if pre is None else pre.data_ptr(),
                    2 * n_out)
    if ws is None:
        ws = _workspace(_size("vb_gated_linear_forward_workspace", p), x.device)
    _run("vb_gated_linear_forward", p, *_scratch(ws, dev), _stream(dev))
    return (y, pre) if want_pre else y


def gated_linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, pre: torch.Tensor,
                          act: str = "silu", want_x: bool = True, want_weight: bool = True, want_bias: bool = True,
                          ws: Optional[torch.Tensor] = None, round_g: bool = False):
    """Gradients of `gated_linear` (vb_gated_linear_backward) for the gradient dy of y and the forward
    pass's pre: (dx, dweight, dbias), None where not wanted.  round_g: in a 16-bit type, dx and dweight
    from the gradient of pre rounded to the type, in about half the time."""
    dev = _device(x)
    dt = _dtype(x)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    rows, n_in = x.shape
    n_out = _halves(weight)
    _no_graph(dy, x, weight, pre)
    ld_dy = _matrix("dy", dy, rows, n_out, x)
    ld_x = _matrix("x", x, rows, n_in, x)
    ld_w = _matrix("weight", weight, 2 * n_out, n_in, x)
    ld_p = _matrix("pre", pre, rows, 2 * n_out, x)
    dx = x.new_empty((rows, n_in)) if want_x else None
    dw = x.new_empty((2 * n_out, n_in)) if want_weight else None
    db = x.new_empty((2 * n_out,)) if want_bias else None
    p = _GATED_BWD.pack(rows, n_in, n_out, dt, _act(act), dy.data_ptr(), ld_dy, x.data_ptr(), ld_x, weight.data_ptr(),
                        ld_w, pre.data_ptr(), ld_p, 0 if dx is None else dx.data_ptr(), n_in,
                        0 if dw is None else dw.data_ptr(), n_in, 0 if db is None else db.data_ptr(), bool(round_g))
    if ws is None:
        ws = _workspace(_size("vb_gated_linear_backward_workspace", p), x.device)
    _run("vb_gated_linear_backward", p, *_scratch(ws, dev), _stream(dev))
    return dx, dw, db


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, want_stats: bool = False, out: Optional[torch.Tensor] = None):
    """y = (x - mean) rstd weight + bias of each row of x [rows][n] (vb_layer_norm_forward), rstd =
    1 / sqrt(variance + eps); weight and bias [n].  With want_stats also the rows' statistics in
    float32, which layer_norm_backward needs: (y, mean, rstd).  `out` may be x itself."""
    dev = _device(x)
    dt = _dtype(x)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    rows, n = x.shape
    _no_graph(x, weight, bias, out)
    ld_x = _matrix("x", x, rows, n, x)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _vector(name, t, n, x)
    if out is None:
        y, ld_y = x.new_empty((rows, n)), n
    else:
        y, ld_y = out, _matrix("out", out, rows, n, x)
    mean = x.new_empty(rows, dtype=torch.float32) if want_stats else None
    rstd = x.new_empty(rows, dtype=torch.float32) if want_stats else None
    p = _NORM.pack(rows, n, dt, x.data_ptr(), ld_x, 0 if weight is None else weight.data_ptr(),
                   0 if bias is None else bias.data_ptr(), eps, y.data_ptr(), ld_y,
                   0 if mean is None else mean.data_ptr(), 0 if rstd is None else rstd.data_ptr())
    _run("vb_layer_norm_forward", p, _stream(dev))
    return (y, mean, rstd) if want_stats else y


def layer_norm_workspace(x: torch.Tensor) -> torch.Tensor:
    """A workspace for `layer_norm_backward` calls of these sizes, to keep between calls."""
    _device(x)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    return _workspace(_size("vb_layer_norm_backward_workspace", *x.shape, _dtype(x)), x.device)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, dresidual: Optional[torch.Tensor] = None,
                        want_x: bool = True, want_weight: bool = True, want_bias: bool = True,
                        dx: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Gradients of `layer_norm` (vb_layer_norm_backward) for the gradient dy of y and the forward pass's
    statistics: (dx, dweight, dbias), None where not wanted.  dresidual: the gradient that reaches x
    past the norm, added to dx.  `dx` may be dy or dresidual itself."""
    dev = _device(x)
    dt = _dtype(x)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    rows, n = x.shape
    _no_graph(dy, x, mean, rstd, weight, dresidual, dx)
    ld_x = _matrix("x", x, rows, n, x)
    ld_dy = _matrix("dy", dy, rows, n, x)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype is not torch.float32 or t.shape != (rows,) or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 [{rows}] on {x.device}")
    if weight is not None:
        _vector("weight", weight, n, x)
    ld_r = n if dresidual is None else _matrix("dresidual", dresidual, rows, n, x)
    ld_dx = n
    if dx is not None:
        ld_dx = _matrix("dx", dx, rows, n, x)
    elif want_x:
        dx = x.new_empty((rows, n))
    dw = x.new_empty((n,)) if want_weight else None
    db = x.new_empty((n,)) if want_bias else None
    if ws is None:
        ws = layer_norm_workspace(x)
    p = _NORM_BWD.pack(rows, n, dt, dy.data_ptr(), ld_dy, x.data_ptr(), ld_x, mean.data_ptr(), rstd.data_ptr(),
                       0 if weight is None else weight.data_ptr(), 0 if dresidual is None else dresidual.data_ptr(),
                       ld_r, 0 if dx is None else dx.data_ptr(), ld_dx, 0 if dw is None else dw.data_ptr(),
                       0 if db is None else db.data_ptr())
    _run("vb_layer_norm_backward", p, *_scratch(ws, dev), _stream(dev))
    return dx, dw, db


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, residual: Optional[torch.Tensor] = None,
            step: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dropout of x [rows][n] with the mask that (seed, offset) give (vb_dropout): kept elements / (1 - p),
    zeros elsewhere, + residual.  The backward pass is the same call on the gradient, without the
    residual.  seed and offset: 64-bit numbers, another offset for each use.  step: an int64 [1] on the
    GPU that is added to offset, for calls that are captured and replayed.  `out` may be x or the
    residual itself."""
    dev = _device(x)
    dt = _dtype(x)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    if not 0 <= seed < 2 ** 64 or not 0 <= offset < 2 ** 64:
        raise ValueError(f"seed and offset must be in [0, 2^64), got {seed} and {offset}")
    rows, n = x.shape
    _no_graph(x, residual, out)
    ld_x = _matrix("x", x, rows, n, x)
    ld_r = n if residual is None else _matrix("residual", residual, rows, n, x)
    if step is not None and (step.dtype is not torch.int64 or step.shape != (1,) or step.get_device() != dev):
        raise ValueError(f"step must be int64 [1] on {x.device}")
    if out is None:
        y, ld_y = x.new_empty((rows, n)), n
    else:
        y, ld_y = out, _matrix("out", out, rows, n, x)
    a = _DROP.pack(rows, n, dt, x.data_ptr(), ld_x, 0 if residual is None else residual.data_ptr(), ld_r, p, seed, offset,
                   0 if step is None else step.data_ptr(), y.data_ptr(), ld_y)
    _run("vb_dropout", a, _stream(dev))
    return y
