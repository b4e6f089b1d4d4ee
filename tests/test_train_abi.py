"""The training operators reject bad arguments on the host, before any launch (fake
device addresses: nothing is dereferenced), and the binding refuses wrong tensors."""
import ctypes

import pytest
import torch

from helpers import ensure_built

ensure_built()
import linear_bound_propagation_amd as lbp  # noqa: E402
from linear_bound_propagation_amd import train  # noqa: E402

L = lbp.lib()
P = ctypes.c_void_p
EINVAL, ESHAPE, ENOMEM = -1, -2, -3


def message():
    return L.vb_last_error().decode()


def size(fn, *args):
    out = ctypes.c_size_t(0)
    return fn(*args, ctypes.byref(out)), out.value


def fwd(**kw):
    d = dict(rows=8, n_in=12, n_out=10, dtype=0, act=0, x=4096, ld_x=12, weight=8192, ld_w=12, y=12288, ld_y=10)
    d.update(kw)
    return L.vb_linear_forward(ctypes.byref(train.vb_linear_fwd(**d)), None, 0, None)


def test_linear_forward_refusals():
    assert L.vb_linear_forward(None, None, 0, None) == EINVAL
    for kw, want, text in (
            (dict(rows=-1), EINVAL, "rows"), (dict(rows=2 ** 31), EINVAL, "rows"), (dict(n_in=0), EINVAL, "sizes"),
            (dict(n_out=-3), EINVAL, "sizes"), (dict(n_in=2 ** 20 + 1), -5, "not supported"), (dict(dtype=3), EINVAL, "dtype"), (dict(dtype=-1), EINVAL, "dtype"),
            (dict(act=4), EINVAL, "activation"), (dict(x=None), EINVAL, "x is NULL"),
            (dict(weight=None), EINVAL, "weight is NULL"), (dict(y=None), EINVAL, "y is NULL"),
            (dict(x=4098), EINVAL, "aligned"), (dict(dtype=1, bias=4097), EINVAL, "bias is not aligned"),
            (dict(ld_x=11), ESHAPE, "leading dimension of x"), (dict(ld_w=0), ESHAPE, "of weight"),
            (dict(ld_y=9), ESHAPE, "of y"), (dict(residual=512, ld_res=3), ESHAPE, "of residual"),
            (dict(residual=512, ld_res=0), ESHAPE, "of residual"), (dict(pre=512, ld_pre=9), ESHAPE, "of pre"),
            (dict(ld_x=2 ** 30 + 1), ESHAPE, "leading dimension"),
            (dict(residual=12288, ld_res=11), ESHAPE, "same leading dimension")):
        assert fwd(**kw) == want, kw
        assert text in message() and "vb_linear_forward" in message(), (kw, message())
    assert fwd(rows=0, x=None, y=None) == 0         # nothing to do


def bwd(ws=65536, ws_bytes=1 << 30, **kw):
    d = dict(rows=8, n_in=12, n_out=10, dtype=0, act=1, dy=4096, ld_dy=10, x=8192, ld_x=12, weight=12288, ld_w=12,
             saved=16384, ld_saved=10, dx=20480, ld_dx=12, dweight=24576, ld_dw=12, dbias=28672, dresidual=32768,
             ld_dres=10)
    d.update(kw)
    return L.vb_linear_backward(ctypes.byref(train.vb_linear_bwd(**d)), ws, ws_bytes, None)


def test_linear_backward_refusals():
    assert L.vb_linear_backward(None, None, 0, None) == EINVAL
    for kw, want, text in (
            (dict(rows=-1), EINVAL, "rows"), (dict(n_in=0), EINVAL, "sizes"), (dict(dtype=7), EINVAL, "dtype"),
            (dict(act=-1), EINVAL, "activation"), (dict(dy=None), EINVAL, "dy is NULL"),
            (dict(x=None), EINVAL, "x is NULL"), (dict(weight=None), EINVAL, "weight is NULL"),
            (dict(saved=None), EINVAL, "saved is NULL"), (dict(ld_saved=9), ESHAPE, "of saved"),
            (dict(ld_dx=11), ESHAPE, "of dx"), (dict(ld_dw=11), ESHAPE, "of dweight"),
            (dict(ld_dres=9), ESHAPE, "of dresidual"), (dict(ld_dy=0), ESHAPE, "of dy"),
            (dict(dx=None, dweight=None, dbias=None, dresidual=None), EINVAL, "nothing to compute"),
            (dict(dresidual=4096, ld_dres=12), ESHAPE, "same leading dimension"),
            (dict(ws=None), ENOMEM, "workspace too small"), (dict(ws_bytes=8), ENOMEM, "workspace too small"),
            (dict(ws=65540), EINVAL, "16-byte aligned")):
        assert bwd(**kw) == want, kw
        assert text in message() and "vb_linear_backward" in message(), (kw, message())


def test_linear_workspace():
    def need(fn, cls, **kw):
        d = dict(rows=100, n_in=64, n_out=40, dtype=0, act=1, x=4096, ld_x=64, weight=8192, ld_w=64)
        if cls is train.vb_linear_bwd:
            d.update(dy=4096, ld_dy=40, dx=16, dweight=16, dbias=16)
        d.update(kw)
        return size(fn, ctypes.byref(cls(**d)))

    fwd, bwd = (L.vb_linear_forward_workspace, train.vb_linear_fwd), (L.vb_linear_backward_workspace, train.vb_linear_bwd)
    for fn, cls in (fwd, bwd):
        assert need(fn, cls)[0] == 0 and need(fn, cls, rows=0) == (0, 0)
        assert fn(None, ctypes.byref(ctypes.c_size_t(0))) == EINVAL
        assert fn(ctypes.byref(cls(rows=1, n_in=1, n_out=1)), None) == EINVAL
        assert need(fn, cls, rows=-8)[0] == EINVAL and need(fn, cls, dtype=9)[0] == EINVAL
        assert need(fn, cls, n_in=2 ** 20 + 1)[0] == -5
        # rows that a large product cannot read are copied
        base = need(fn, cls)[1]
        assert need(fn, cls, x=4100)[1] >= base + 100 * 64 * 4
        assert need(fn, cls, ld_w=65)[1] >= base + 40 * 64 * 4
        assert need(fn, cls, n_in=63)[1] >= base
    assert need(*fwd, rows=5, x=4100)[1] == 0          # few rows: no copy
    st, n = need(*bwd, rows=2 ** 31 - 1, n_in=8192, n_out=16384, dtype=1, ld_x=8192, ld_w=8192, ld_dy=16384)
    assert st == 0 and n >= (2 ** 31 - 1) * 16384 * 2   # no 32-bit overflow


def loss(ws=65536, ws_bytes=1 << 20, **kw):
    d = dict(rows=8, classes=10, dtype=0, logits=4096, ld=10, labels=8192, ignore_index=-100, label_smoothing=0.0,
             grad_scale=1.0, loss=12288, row_loss=16384, dlogits=20480, ld_d=10)
    d.update(kw)
    return L.vb_cross_entropy(ctypes.byref(train.vb_cross_entropy_args(**d)), ws, ws_bytes, None)


def test_cross_entropy_refusals():
    assert L.vb_cross_entropy(None, None, 0, None) == EINVAL
    for kw, want, text in (
            (dict(rows=-1), EINVAL, "rows"), (dict(classes=0), EINVAL, "sizes"), (dict(dtype=3), EINVAL, "dtype"),
            (dict(logits=None), EINVAL, "logits is NULL"), (dict(labels=None), EINVAL, "labels is NULL"),
            (dict(labels=8196), EINVAL, "labels is not aligned"), (dict(loss=12290), EINVAL, "not aligned"),
            (dict(ld=9), ESHAPE, "of logits"), (dict(ld_d=9), ESHAPE, "of dlogits"),
            (dict(label_smoothing=-0.1), EINVAL, "label_smoothing"),
            (dict(label_smoothing=1.5), EINVAL, "label_smoothing"),
            (dict(label_smoothing=float("nan")), EINVAL, "label_smoothing"),
            (dict(loss=None, row_loss=None, dlogits=None), EINVAL, "nothing to compute"),
            (dict(dlogits=4096, ld_d=12), ESHAPE, "same leading dimension"),
            (dict(ws=None), ENOMEM, "workspace too small"), (dict(ws_bytes=4), ENOMEM, "workspace too small"),
            (dict(ws=65544), EINVAL, "16-byte aligned")):
        assert loss(**kw) == want, kw
        assert text in message() and "vb_cross_entropy" in message(), (kw, message())
    assert L.vb_cross_entropy_workspace(8, 10, 0, None) == EINVAL
    assert size(L.vb_cross_entropy_workspace, 8, 0, 0)[0] == EINVAL


def clip(n=2, grads=(4096, 8192), out=None, sizes=(10, 20), dtypes=(0, 1), max_norm=1.0, norm=12288, ws=65536,
         ws_bytes=1 << 20):
    g = None if grads is None else (P * 2)(*grads)
    o = None if out is None else (P * 2)(*out)
    s = None if sizes is None else (ctypes.c_int64 * 2)(*sizes)
    d = None if dtypes is None else (ctypes.c_int32 * 2)(*dtypes)
    return L.vb_clip_grad_norm(n, g, o, s, d, max_norm, norm, ws, ws_bytes, None)


def test_clip_refusals():
    for kw, want, text in (
            (dict(n=-1), EINVAL, "tensor list"), (dict(grads=None), EINVAL, "tensor list"),
            (dict(sizes=None), EINVAL, "tensor list"), (dict(dtypes=None), EINVAL, "tensor list"),
            (dict(norm=None), EINVAL, "norm"), (dict(norm=12290), EINVAL, "norm"),
            (dict(max_norm=-1.0), EINVAL, "max_norm"), (dict(max_norm=float("nan")), EINVAL, "max_norm"),
            (dict(sizes=(10, -1)), EINVAL, "negative"), (dict(dtypes=(0, 5)), EINVAL, "dtype 5 of tensor 1"),
            (dict(grads=(4096, None)), EINVAL, "tensor 1"), (dict(grads=(4098, 8192)), EINVAL, "tensor 0"),
            (dict(out=(4096, None)), EINVAL, "tensor 1"), (dict(ws=None), ENOMEM, "workspace too small"),
            (dict(ws_bytes=8), ENOMEM, "workspace too small"), (dict(ws=65544), EINVAL, "16-byte aligned")):
        assert clip(**kw) == want, kw
        assert text in message() and "vb_clip_grad_norm" in message(), (kw, message())
    assert L.vb_clip_grad_norm_workspace(1, None, None) == EINVAL
    assert size(L.vb_clip_grad_norm_workspace, 0, None)[0] == 0


def test_the_binding_refuses_host_tensors_and_wrong_types():
    x, w = torch.zeros(4, 3), torch.zeros(5, 3)
    for call in (lambda: lbp.linear(x, w), lambda: lbp.linear_backward(torch.zeros(4, 5), x, w),
                 lambda: lbp.cross_entropy(x, torch.zeros(4, dtype=torch.int64)),
                 lambda: lbp.clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError, match="current GPU"):
            call()
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        train._dtype(torch.zeros(1, dtype=torch.float64))
    like = torch.zeros(4, 3)
    for bad, text in ((torch.zeros(3, 4), "must be"), (torch.zeros(4, 3, 1), "must be"),
                      (torch.zeros(4, 3, dtype=torch.float16), "must be"), (torch.zeros(3, 4).t(), "contiguous")):
        with pytest.raises(ValueError, match=text):
            train._matrix("x", bad, 4, 3, like)
    assert train._matrix("x", torch.zeros(4, 9)[:, 2:5], 4, 3, like) == 9
    for bad in (torch.zeros(4), torch.zeros(3, 1), torch.zeros(6)[::2], torch.zeros(3, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            train._vector("bias", bad, 3, like)
