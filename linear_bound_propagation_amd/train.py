"""Training and evaluation of the networks whose bounds the package computes:
the fused linear layer and its backward pass, the softmax cross entropy with its
gradient, and the clipping of gradients to a global norm (include/vb_train.h).

Thin ctypes binding, like the rest of the package: every step runs in the
library's HIP kernels on the current stream; results are new tensors on it.
Matrices may have any row stride; elements of a row are contiguous.
"""
from __future__ import annotations

import ctypes
from typing import List, Optional, Sequence, Tuple

import torch

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}

EXPORTS = ["vb_linear_forward_workspace", "vb_linear_backward_workspace", "vb_linear_forward",
           "vb_linear_backward", "vb_cross_entropy_workspace", "vb_cross_entropy", "vb_clip_grad_norm_workspace", "vb_clip_grad_norm"]

_P, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t


class vb_linear_fwd(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n_in", _i32), ("n_out", _i32), ("dtype", _i32), ("act", _i32),
                ("x", _P), ("ld_x", _i64), ("weight", _P), ("ld_w", _i64), ("bias", _P),
                ("residual", _P), ("ld_res", _i64), ("y", _P), ("ld_y", _i64), ("pre", _P), ("ld_pre", _i64)]


class vb_linear_bwd(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n_in", _i32), ("n_out", _i32), ("dtype", _i32), ("act", _i32),
                ("dy", _P), ("ld_dy", _i64), ("x", _P), ("ld_x", _i64), ("weight", _P), ("ld_w", _i64),
                ("saved", _P), ("ld_saved", _i64), ("dx", _P), ("ld_dx", _i64), ("dweight", _P), ("ld_dw", _i64),
                ("dbias", _P), ("dresidual", _P), ("ld_dres", _i64)]


class vb_cross_entropy_args(ctypes.Structure):
    _fields_ = [("rows", _i64), ("classes", _i32), ("dtype", _i32), ("logits", _P), ("ld", _i64), ("labels", _P),
                ("ignore_index", _i64), ("label_smoothing", _f32), ("grad_scale", _f32), ("loss", _P),
                ("row_loss", _P), ("dlogits", _P), ("ld_d", _i64)]


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the calls of vb_train.h."""
    psz = ctypes.POINTER(_sz)
    for name, args in (("vb_linear_forward_workspace", [ctypes.POINTER(vb_linear_fwd), psz]),
                       ("vb_linear_backward_workspace", [ctypes.POINTER(vb_linear_bwd), psz]),
                       ("vb_linear_forward", [ctypes.POINTER(vb_linear_fwd), _P, _sz, _P]),
                       ("vb_linear_backward", [ctypes.POINTER(vb_linear_bwd), _P, _sz, _P]),
                       ("vb_cross_entropy_workspace", [_i64, _i32, _i32, psz]),
                       ("vb_cross_entropy", [ctypes.POINTER(vb_cross_entropy_args), _P, _sz, _P]),
                       ("vb_clip_grad_norm_workspace", [_i32, ctypes.POINTER(_i64), psz]),
                       ("vb_clip_grad_norm", [_i32, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_i64),
                                              ctypes.POINTER(_i32), _f32, _P, _P, _sz, _P])):
        fn = getattr(lib, name)
        fn.restype = _i32
        fn.argtypes = args


def _pkg():
    import linear_bound_propagation_amd as pkg
    return pkg


def _dtype(t: torch.Tensor) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"float32, bfloat16 or float16 expected, got {t.dtype}")
    return code


def _matrix(name: str, t: torch.Tensor, rows: int, cols: int, like: torch.Tensor) -> int:
    """Leading dimension of a [rows][cols] operand (checked against `like`'s type and device)."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} must be [{rows}][{cols}], got {tuple(t.shape)}")
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"the elements of a row of {name} must be contiguous")
    return t.stride(0) if rows > 1 else max(cols, t.stride(0))


def _vector(name: str, t: torch.Tensor, n: int, like: torch.Tensor) -> None:
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}], got {tuple(t.shape)}")
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")


def _device(t: torch.Tensor) -> None:
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current GPU, got {t.device}")


def _bytes(n: int, device) -> Optional[torch.Tensor]:
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _workspace(ws: Optional[torch.Tensor], need: int, device):
    """(pointer, bytes, tensor): the caller's workspace, or a new one of `need` bytes."""
    if ws is None:
        ws = _bytes(need, device)
    return (None, 0, None) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size(), ws)


def _size(fn: str, *args) -> int:
    pkg = _pkg()
    out = _sz(0)
    pkg._check(getattr(pkg.lib(), fn)(*args, ctypes.byref(out)), fn)
    return out.value


def linear_workspace(x: torch.Tensor, weight: torch.Tensor, backward: bool = False) -> torch.Tensor:
    """A workspace for `linear` calls (or `linear_backward` calls, with any activation and all
    gradients) on tensors of these sizes and strides, to keep between calls."""
    _device(x)
    rows, n_in = x.shape
    n_out = weight.shape[0]
    ld_x, ld_w = _matrix("x", x, rows, n_in, x), _matrix("weight", weight, n_out, n_in, x)
    if backward:
        p = vb_linear_bwd(rows, n_in, n_out, _dtype(x), ACTS["silu"], None, n_out, x.data_ptr(), ld_x,
                          weight.data_ptr(), ld_w, None, n_out, 16, n_in, 16, n_in, 16, 16, n_out)
        n = _size("vb_linear_backward_workspace", ctypes.byref(p))
    else:
        p = vb_linear_fwd(rows, n_in, n_out, _dtype(x), 0, x.data_ptr(), ld_x, weight.data_ptr(), ld_w)
        n = _size("vb_linear_forward_workspace", ctypes.byref(p))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
           residual: Optional[torch.Tensor] = None, act: str = "none", want_pre: bool = False,
           out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """y = act(x W^T + bias + residual) (vb_linear_forward): x [rows][n_in], weight
    [n_out][n_in], bias [n_out], residual [rows][n_out]; act one of none, relu, gelu, silu.
    With want_pre also the value before the activation, which linear_backward needs for
    gelu and silu: (y, pre).  `out` may be the residual itself."""
    pkg = _pkg()
    _device(x)
    dt = _dtype(x)
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x and weight must be matrices")
    rows, n_in = x.shape
    n_out = weight.shape[0]
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    ld_x = _matrix("x", x, rows, n_in, x)
    ld_w = _matrix("weight", weight, n_out, n_in, x)
    if bias is not None:
        _vector("bias", bias, n_out, x)
    ld_res = 0 if residual is None else _matrix("residual", residual, rows, n_out, x)
    y = torch.empty(rows, n_out, dtype=x.dtype, device=x.device) if out is None else out
    ld_y = n_out if out is None else _matrix("out", out, rows, n_out, x)
    pre = torch.empty(rows, n_out, dtype=x.dtype, device=x.device) if want_pre else None
    p = vb_linear_fwd(rows, n_in, n_out, dt, ACTS[act], x.data_ptr(), ld_x, weight.data_ptr(), ld_w,
                      None if bias is None else bias.data_ptr(), None if residual is None else residual.data_ptr(),
                      ld_res, y.data_ptr(), ld_y, None if pre is None else pre.data_ptr(), n_out)
    wp, wn, keep = _workspace(ws, _size("vb_linear_forward_workspace", ctypes.byref(p)) if ws is None else 0, x.device)
    pkg._check(pkg.lib().vb_linear_forward(ctypes.byref(p), wp, wn, pkg._stream()), "vb_linear_forward")
    return (y, pre) if want_pre else y


def linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, act: str = "none",
                    saved: Optional[torch.Tensor] = None, want_x: bool = True, want_weight: bool = True,
                    want_bias: bool = True, want_residual: bool = False, ws: Optional[torch.Tensor] = None):
    """Gradients of `linear` (vb_linear_backward) for the gradient dy of y: (dx, dweight, dbias,
    dresidual), None where not wanted.  saved: y for relu, pre for gelu and silu."""
    pkg = _pkg()
    _device(x)
    dt = _dtype(x)
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x and weight must be matrices")
    rows, n_in = x.shape
    n_out = weight.shape[0]
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    if (saved is None) != (act == "none"):
        raise ValueError("saved is the forward pass's y (relu) or pre (gelu, silu), and None without an activation")
    ld_dy = _matrix("dy", dy, rows, n_out, x)
    ld_x = _matrix("x", x, rows, n_in, x)
    ld_w = _matrix("weight", weight, n_out, n_in, x)
    ld_s = 0 if saved is None else _matrix("saved", saved, rows, n_out, x)

    def new(want, *shape):
        return torch.empty(shape, dtype=x.dtype, device=x.device) if want else None

    dx, dw, db, dr = (new(want_x, rows, n_in), new(want_weight, n_out, n_in), new(want_bias, n_out),
                      new(want_residual, rows, n_out))
    p = vb_linear_bwd(rows, n_in, n_out, dt, ACTS[act], dy.data_ptr(), ld_dy, x.data_ptr(), ld_x, weight.data_ptr(),
                      ld_w, None if saved is None else saved.data_ptr(), ld_s, None if dx is None else dx.data_ptr(),
                      n_in, None if dw is None else dw.data_ptr(), n_in, None if db is None else db.data_ptr(),
                      None if dr is None else dr.data_ptr(), n_out)
    wp, wn, keep = _workspace(ws, _size("vb_linear_backward_workspace", ctypes.byref(p)) if ws is None else 0, x.device)
    pkg._check(pkg.lib().vb_linear_backward(ctypes.byref(p), wp, wn, pkg._stream()), "vb_linear_backward")
    return dx, dw, db, dr


def cross_entropy_workspace(logits: torch.Tensor) -> torch.Tensor:
    """A workspace for `cross_entropy` calls of these sizes, to keep between calls."""
    return _bytes(_size("vb_cross_entropy_workspace", logits.shape[0], logits.shape[1], _dtype(logits)), logits.device)


def cross_entropy(logits: torch.Tensor, labels: torch.Tensor, ignore_index: int = -100,
                  label_smoothing: float = 0.0, grad_scale: float = 1.0, want_grad: bool = True,
                  dlogits: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Softmax cross entropy of labels [rows] (int64) and its gradient (vb_cross_entropy): (loss [1],
    row_loss [rows], dlogits [rows][classes] or None).  loss is the mean over the rows whose label
    is not ignore_index; `dlogits` may be the logits themselves."""
    pkg = _pkg()
    _device(logits)
    dt = _dtype(logits)
    if logits.dim() != 2:
        raise ValueError("logits must be a matrix")
    rows, classes = logits.shape
    ld = _matrix("logits", logits, rows, classes, logits)
    if labels.dtype != torch.int64 or labels.shape != (rows,) or labels.device != logits.device \
            or not labels.is_contiguous():
        raise ValueError(f"labels must be contiguous int64 [{rows}] on {logits.device}")
    if dlogits is None:
        ld_d = classes
        if want_grad:
            dlogits = torch.empty(rows, classes, dtype=logits.dtype, device=logits.device)
    else:
        ld_d = _matrix("dlogits", dlogits, rows, classes, logits)
    both = torch.empty(rows + 1, dtype=torch.float32, device=logits.device)
    base = both.data_ptr()
    wp, wn, keep = _workspace(ws, _size("vb_cross_entropy_workspace", rows, classes, dt) if ws is None else 0,
                              logits.device)
    p = vb_cross_entropy_args(rows, classes, dt, logits.data_ptr(), ld, labels.data_ptr(), ignore_index,
                              label_smoothing, grad_scale, base + 4 * rows, base,
                              None if dlogits is None else dlogits.data_ptr(), ld_d)
    pkg._check(pkg.lib().vb_cross_entropy(ctypes.byref(p), wp, wn, pkg._stream()), "vb_cross_entropy")
    return both[rows:], both[:rows], dlogits


def _clip_arrays(grads: Sequence[torch.Tensor]):
    n = len(grads)
    return n, (_i64 * max(n, 1))(*[g.numel() for g in grads])


def clip_grad_norm_workspace(grads: Sequence[torch.Tensor]) -> torch.Tensor:
    """A workspace for `clip_grad_norm` calls on tensors of these sizes, to keep between calls."""
    return _bytes(_size("vb_clip_grad_norm_workspace", *_clip_arrays(grads)), grads[0].device if grads else "cuda")


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
                   ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, List[torch.Tensor]]:
    """Global norm of the gradients, and the gradients clipped to max_norm (vb_clip_grad_norm):
    (norm [1] float32, out).  In place without `out`; a norm that is not finite clips nothing.
    Tensors are contiguous, of any mix of the three types."""
    pkg = _pkg()
    n, sizes = _clip_arrays(grads)
    dev = grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
    if dev.type != "cuda" or dev.index != torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current GPU, got {dev}")
    if out is not None and len(out) != n:
        raise ValueError(f"{len(out)} outputs for {n} gradients")
    for i, g in enumerate(grads):
        if not g.is_contiguous() or g.device != dev:
            raise ValueError(f"gradient {i} must be contiguous, on {dev}")
        if out is not None:
            o = out[i]
            if o.shape != g.shape or o.dtype != g.dtype or o.device != dev or not o.is_contiguous():
                raise ValueError(f"output {i} must be like its gradient: contiguous {g.dtype} {tuple(g.shape)} on {dev}")
    dts = (_i32 * max(n, 1))(*[_dtype(g) for g in grads])
    src = (_P * max(n, 1))(*[g.data_ptr() for g in grads])
    dst = None if out is None else (_P * max(n, 1))(*[o.data_ptr() for o in out])
    norm = torch.empty(1, dtype=torch.float32, device=dev)
    wp, wn, keep = _workspace(ws, _size("vb_clip_grad_norm_workspace", n, sizes) if ws is None else 0, dev)
    pkg._check(pkg.lib().vb_clip_grad_norm(n, src, dst, sizes, dts, max_norm, norm.data_ptr(), wp, wn, pkg._stream()),
               "vb_clip_grad_norm")
    return norm, list(grads if out is None else out)
