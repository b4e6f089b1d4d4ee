"""The gated linear layer, layer norm and dropout reject bad arguments on the host, before any
launch (fake device addresses: nothing is dereferenced), and the binding refuses wrong tensors."""
import ctypes
import math

import pytest
import torch

from helpers import ensure_built

ensure_built()
import linear_bound_propagation_amd as lbp  # noqa: E402
from linear_bound_propagation_amd import train  # noqa: E402

L = lbp.lib()
EINVAL, ESHAPE, ENOMEM, EUNSUPPORTED = -1, -2, -3, -5


def message():
    return L.vb_last_error().decode()


def refused(fn, name, table):
    for kw, want, text in table:
        assert fn(**kw) == want, (kw, message())
        assert text in message() and name in message(), (kw, message())


def size(fn, *args):
    out = ctypes.c_size_t(0)
    return fn(*args, ctypes.byref(out)), out.value


def gated(ws=1 << 22, ws_bytes=1 << 30, **kw):
    d = dict(rows=80, n_in=12, n_out=10, dtype=0, act=3, x=1 << 12, ld_x=12, weight=1 << 14, ld_w=12, y=1 << 16, ld_y=10)
    d.update(kw)
    return L.vb_gated_linear_forward(ctypes.byref(train.vb_gated_linear_fwd(**d)), ws, ws_bytes, None)


def test_gated_refusals():
    assert L.vb_gated_linear_forward(None, None, 0, None) == EINVAL
    refused(gated, "vb_gated_linear_forward", (
        (dict(rows=-1), EINVAL, "rows"), (dict(rows=2 ** 31), EINVAL, "rows"), (dict(n_in=0), EINVAL, "sizes"),
        (dict(n_out=0), EINVAL, "sizes"), (dict(n_in=2 ** 20 + 1), EUNSUPPORTED, "not supported"),
        (dict(n_out=2 ** 19 + 1), EUNSUPPORTED, "n_out above"), (dict(n_out=2 ** 31 - 1), EUNSUPPORTED, "not supported"),
        (dict(dtype=3), EINVAL, "dtype"), (dict(act=4), EINVAL, "activation"), (dict(act=-1), EINVAL, "activation"),
        (dict(x=None), EINVAL, "x is NULL"), (dict(weight=None), EINVAL, "weight is NULL"), (dict(y=None), EINVAL, "y is NULL"),
        (dict(x=4098), EINVAL, "aligned"), (dict(ld_x=11), ESHAPE, "of x"), (dict(ld_w=11), ESHAPE, "of weight"),
        (dict(ld_y=9), ESHAPE, "of y"), (dict(pre=1 << 18, ld_pre=19), ESHAPE, "of pre"),
        (dict(dtype=1, bias=4097), EINVAL, "bias is not aligned"), (dict(ws=None, ld_x=17), ENOMEM, "workspace"),
        (dict(ws_bytes=64, ld_x=17), ENOMEM, "workspace"), (dict(ws=(1 << 22) + 8, ld_x=17), EINVAL, "16-byte"),
        (dict(y=1 << 12), EINVAL, "y overlaps x"), (dict(y=(1 << 14) + 10 * 48), EINVAL, "y overlaps weight"),
        (dict(pre=(1 << 16) + 40, ld_pre=20), EINVAL, "overlaps"), (dict(bias=1 << 16), EINVAL, "y overlaps bias"),
        (dict(bias=(1 << 16) - 40), EINVAL, "y overlaps bias"),             # its last number
        (dict(ws=1 << 16, ld_x=17), EINVAL, "overlaps")))
    assert gated(rows=0, x=None, weight=None, y=None, ws=None, ws_bytes=0) == 0


def gated_back(ws=1 << 22, ws_bytes=1 << 30, **kw):
    d = dict(rows=8, n_in=12, n_out=10, dtype=0, act=3, dy=1 << 12, ld_dy=10, x=1 << 13, ld_x=12, weight=1 << 14, ld_w=12,
             pre=1 << 15, ld_pre=20, dx=1 << 16, ld_dx=12, dweight=1 << 17, ld_dw=12, dbias=1 << 18)
    d.update(kw)
    return L.vb_gated_linear_backward(ctypes.byref(train.vb_gated_linear_bwd(**d)), ws, ws_bytes, None)


def test_gated_backward_refusals():
    assert L.vb_gated_linear_backward(None, None, 0, None) == EINVAL
    refused(gated_back, "vb_gated_linear_backward", (
        (dict(rows=-1), EINVAL, "rows"), (dict(n_out=2 ** 19 + 1), EUNSUPPORTED, "n_out above"), (dict(act=9), EINVAL, "activation"),
        (dict(round_g=2), EINVAL, "round_g"), (dict(dy=None), EINVAL, "dy is NULL"), (dict(x=None), EINVAL, "x is NULL"),
        (dict(weight=None), EINVAL, "weight is NULL"), (dict(pre=None), EINVAL, "pre is NULL"), (dict(ld_pre=19), ESHAPE, "of pre"),
        (dict(ld_dy=9), ESHAPE, "of dy"), (dict(ld_dx=11), ESHAPE, "of dx"), (dict(ld_dw=11), ESHAPE, "of dweight"),
        (dict(dx=None, dweight=None, dbias=None), EINVAL, "nothing to compute"), (dict(ws=None), ENOMEM, "workspace"),
        (dict(ws_bytes=100), ENOMEM, "workspace"), (dict(dx=1 << 12), EINVAL, "dx overlaps dy"),
        (dict(dx=(1 << 15) + 76), EINVAL, "dx overlaps pre"), (dict(dbias=(1 << 17) + 19 * 48), EINVAL, "overlaps"),
        (dict(dweight=(1 << 14) - 4), EINVAL, "dweight overlaps weight"), (dict(ws=1 << 15), EINVAL, "workspace overlaps pre")))


def test_gated_workspaces():
    def need(fn, cls, **kw):
        d = dict(rows=100, n_in=64, n_out=40, dtype=1, act=3, x=4096, ld_x=64, weight=8192, ld_w=64)
        if cls is train.vb_gated_linear_bwd:
            d.update(dx=16, dweight=16, dbias=16)
        d.update(kw)
        return size(fn, ctypes.byref(cls(**d)))

    fwd = (L.vb_gated_linear_forward_workspace, train.vb_gated_linear_fwd)
    bwd = (L.vb_gated_linear_backward_workspace, train.vb_gated_linear_bwd)
    for fn, cls in (fwd, bwd):
        assert need(fn, cls)[0] == 0 and need(fn, cls, rows=0) == (0, 0)
        assert fn(None, ctypes.byref(ctypes.c_size_t(0))) == EINVAL and fn(ctypes.byref(cls(rows=1, n_in=1, n_out=1)), None) == EINVAL
        assert need(fn, cls, rows=-8)[0] == EINVAL and need(fn, cls, dtype=9)[0] == EINVAL
        assert need(fn, cls, n_out=2 ** 19 + 1)[0] == EUNSUPPORTED and need(fn, cls, n_out=2 ** 19)[0] == 0
    # unaligned rows are copied: 100 rows of 64 and 80 of weight
    assert need(*fwd, ld_x=65)[1] - need(*fwd)[1] >= 100 * 128
    assert need(*fwd, weight=8194)[1] - need(*fwd)[1] >= 80 * 128
    # g, in two parts without round_g
    one, two = need(*bwd, round_g=1)[1], need(*bwd)[1]
    assert two - one >= 100 * 160 and one >= 100 * 160


def norm(**kw):
    d = dict(rows=8, n=12, dtype=0, x=1 << 12, ld_x=12, eps=1e-5, y=1 << 13, ld_y=12)
    d.update(kw)
    return L.vb_layer_norm_forward(ctypes.byref(train.vb_layer_norm_fwd(**d)), None)


def test_norm_refusals():
    assert L.vb_layer_norm_forward(None, None) == EINVAL
    refused(norm, "vb_layer_norm_forward", (
        (dict(rows=-1), EINVAL, "rows"), (dict(n=0), EINVAL, "sizes"), (dict(n=2 ** 20 + 1), EUNSUPPORTED, "not supported"),
        (dict(dtype=5), EINVAL, "dtype"), (dict(eps=-1e-9), EINVAL, "eps"), (dict(eps=math.nan), EINVAL, "eps"),
        (dict(eps=math.inf), EINVAL, "eps"), (dict(x=None), EINVAL, "x is NULL"), (dict(y=None), EINVAL, "y is NULL"),
        (dict(ld_x=11), ESHAPE, "of x"), (dict(ld_y=11), ESHAPE, "of y"), (dict(weight=4097), EINVAL, "weight is not aligned"),
        (dict(mean=4098), EINVAL, "mean is not aligned"), (dict(rstd=4097), EINVAL, "rstd is not aligned"),
        (dict(y=1 << 12, ld_y=13), ESHAPE, "same leading dimension"), (dict(y=(1 << 12) + 4), EINVAL, "y overlaps x"),
        (dict(weight=1 << 13), EINVAL, "y overlaps weight"), (dict(bias=(1 << 13) + 40), EINVAL, "y overlaps bias"),
        (dict(mean=(1 << 13) + 4), EINVAL, "y overlaps mean"), (dict(rstd=(1 << 12) + 32), EINVAL, "rstd overlaps x"),
        (dict(mean=1 << 15, rstd=(1 << 15) + 28), EINVAL, "mean overlaps rstd")))
    assert norm(rows=0, x=None, y=None) == 0


def norm_back(ws=1 << 22, ws_bytes=1 << 30, **kw):
    d = dict(rows=8, n=12, dtype=0, dy=1 << 12, ld_dy=12, x=1 << 13, ld_x=12, mean=1 << 14, rstd=1 << 15, weight=1 << 16,
             dx=1 << 17, ld_dx=12, dweight=1 << 18, dbias=1 << 19)
    d.update(kw)
    return L.vb_layer_norm_backward(ctypes.byref(train.vb_layer_norm_bwd(**d)), ws, ws_bytes, None)


def test_norm_backward_refusals():
    assert L.vb_layer_norm_backward(None, None, 0, None) == EINVAL
    refused(norm_back, "vb_layer_norm_backward", (
        (dict(rows=-1), EINVAL, "rows"), (dict(n=2 ** 20 + 1), EUNSUPPORTED, "not supported"), (dict(dy=None), EINVAL, "dy is NULL"),
        (dict(x=None), EINVAL, "x is NULL"), (dict(mean=None), EINVAL, "mean is NULL"), (dict(rstd=None), EINVAL, "rstd is NULL"),
        (dict(x=None, dx=None), EINVAL, "x is NULL"), (dict(ld_dy=11), ESHAPE, "of dy"), (dict(ld_x=0), ESHAPE, "of x"),
        (dict(dresidual=1 << 20, ld_dres=11), ESHAPE, "of dresidual"), (dict(ld_dx=11), ESHAPE, "of dx"),
        (dict(dx=None, dweight=None, dbias=None), EINVAL, "nothing to compute"), (dict(ws=None), ENOMEM, "workspace"),
        (dict(ws_bytes=16), ENOMEM, "workspace"), (dict(ws=(1 << 22) + 4), EINVAL, "16-byte"),
        (dict(dx=1 << 12, ld_dx=13), ESHAPE, "dx over dy"), (dict(dx=1 << 20, dresidual=1 << 20, ld_dres=13), ESHAPE, "dx over dresidual"),
        (dict(dx=(1 << 12) + 4), EINVAL, "dx overlaps dy"), (dict(dx=1 << 13), EINVAL, "dx overlaps x"),
        (dict(dx=1 << 16), EINVAL, "dx overlaps weight"), (dict(dweight=1 << 14), EINVAL, "dweight overlaps mean"),
        (dict(dbias=(1 << 18) + 44), EINVAL, "dweight overlaps dbias"), (dict(ws=1 << 12), EINVAL, "workspace overlaps dy")))
    fn = L.vb_layer_norm_backward_workspace
    assert size(fn, 0, 100, 0) == (0, 0) and size(fn, 5, 100, 0)[1] >= 800
    assert size(fn, 5, 0, 0)[0] == EINVAL and size(fn, 5, 5, 9)[0] == EINVAL and fn(5, 5, 0, None) == EINVAL


def drop(**kw):
    d = dict(rows=8, n=12, dtype=0, x=1 << 12, ld_x=12, p=0.5, seed=1, offset=0, y=1 << 13, ld_y=12)
    d.update(kw)
    return L.vb_dropout(ctypes.byref(train.vb_dropout_args(**d)), None)


def test_dropout_refusals():
    assert L.vb_dropout(None, None) == EINVAL
    refused(drop, "vb_dropout", (
        (dict(rows=-1), EINVAL, "rows"), (dict(n=0), EINVAL, "sizes"), (dict(n=2 ** 30 + 1), EUNSUPPORTED, "not supported"),
        (dict(dtype=-1), EINVAL, "dtype"), (dict(p=-0.1), EINVAL, "p must"), (dict(p=1.0001), EINVAL, "p must"),
        (dict(p=math.nan), EINVAL, "p must"), (dict(x=None), EINVAL, "x is NULL"), (dict(y=None), EINVAL, "y is NULL"),
        (dict(ld_x=11), ESHAPE, "of x"), (dict(residual=1 << 14, ld_res=11), ESHAPE, "of residual"),
        (dict(step=(1 << 14) + 4), EINVAL, "step is not aligned"), (dict(y=1 << 12, ld_y=14), ESHAPE, "y over x"),
        (dict(residual=1 << 13, ld_res=14), ESHAPE, "y over residual"), (dict(y=(1 << 12) - 4), EINVAL, "y overlaps x"),
        (dict(residual=(1 << 13) + 8, ld_res=12), EINVAL, "y overlaps residual"), (dict(step=1 << 13), EINVAL, "y overlaps step")))
    assert drop(rows=0, x=None, y=None) == 0


def test_binding_refuses_wrong_tensors():
    """Tensors off the GPU; the rest of the checks needs one."""
    x, w = torch.zeros(4, 6), torch.zeros(10, 6)
    for call in (lambda: lbp.layer_norm(x), lambda: lbp.layer_norm_backward(x, x, x[:, 0], x[:, 0]), lambda: lbp.dropout(x, 0.5, 1),
                 lambda: lbp.gated_linear(x, w), lambda: lbp.gated_linear_backward(x, x, w, x), lambda: lbp.layer_norm_workspace(x),
                 lambda: lbp.gated_linear_workspace(x, w)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call()
