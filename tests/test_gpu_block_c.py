"""What the C ABI of the block's operators takes and the binding does not pass on: outputs with rows
of their own distance, one statistic without the other."""
import ctypes

import pytest
import torch

import block_reference as ref
from helpers import ensure_built
from train_reference import assert_within

pytestmark = pytest.mark.gpu

P = ctypes.c_void_p
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def stream():
    return P(torch.cuda.current_stream().cuda_stream)


def ok(lbp, status):
    assert status == 0, lbp.lib().vb_last_error()


def framed(rows, n, dtype, pad=5, shift=1):
    """A buffer of sevens and the [rows][n] view of it that is written."""
    buf = torch.full((rows + 2, n + pad), 7.0, dtype=dtype, device="cuda")
    return buf, buf[1:rows + 1, shift:shift + n]


def frame_kept(buf, view):
    view.fill_(7.0)
    return bool((buf == 7.0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", [(1, 40, 33), (3, 64, 2100), (9, 700, 31), (20, 96, 50), (150, 130, 70), (300, 600, 515)], ids=str)
def test_gated_outputs_with_strides(lbp, size, dtype):
    """y, pre, dx and dweight inside larger buffers, rows before and behind them and columns beside
    them left as they were."""
    from linear_bound_propagation_amd import train
    rows, n_in, n_out = size
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(dtype)

    x, w, b, dy = normal(rows, n_in), normal(2 * n_out, n_in, std=n_in ** -0.5), normal(2 * n_out), normal(rows, n_out)
    code, es = train.DTYPES[dtype], x.element_size()
    (yb, y), (pb, pre) = framed(rows, n_out, dtype), framed(rows, 2 * n_out, dtype)
    a = train.vb_gated_linear_fwd(rows=rows, n_in=n_in, n_out=n_out, dtype=code, act=3, x=x.data_ptr(), ld_x=n_in,
                                  weight=w.data_ptr(), ld_w=n_in, bias=b.data_ptr(), y=y.data_ptr(), ld_y=y.stride(0),
                                  pre=pre.data_ptr(), ld_pre=pre.stride(0))
    need = ctypes.c_size_t(0)
    ok(lbp, lbp.lib().vb_gated_linear_forward_workspace(ctypes.byref(a), ctypes.byref(need)))
    ws = torch.empty(need.value + 16, dtype=torch.uint8, device="cuda")
    print(f"gated strided outputs {size} {dtype}", flush=True)
    ok(lbp, lbp.lib().vb_gated_linear_forward(ctypes.byref(a), ws.data_ptr(), need.value, stream()))
    want = ref.gated(x, w, b, "silu")
    assert_within(y, *want["y"], "y")
    assert_within(pre, *want["pre"], "pre")
    keep = pre.clone()
    assert frame_kept(yb, y) and frame_kept(pb, pre)
    (xb, dx), (wb, dw) = framed(rows, n_in, dtype), framed(2 * n_out, n_in, dtype)
    db = torch.empty(2 * n_out, dtype=dtype, device="cuda")
    a = train.vb_gated_linear_bwd(rows=rows, n_in=n_in, n_out=n_out, dtype=code, act=3, dy=dy.data_ptr(), ld_dy=n_out,
                                  x=x.data_ptr(), ld_x=n_in, weight=w.data_ptr(), ld_w=n_in, pre=keep.data_ptr(),
                                  ld_pre=2 * n_out, dx=dx.data_ptr(), ld_dx=dx.stride(0), dweight=dw.data_ptr(),
                                  ld_dw=dw.stride(0), dbias=db.data_ptr())
    ok(lbp, lbp.lib().vb_gated_linear_backward_workspace(ctypes.byref(a), ctypes.byref(need)))
    ws = torch.empty(need.value + 16, dtype=torch.uint8, device="cuda")
    ok(lbp, lbp.lib().vb_gated_linear_backward(ctypes.byref(a), ws.data_ptr(), need.value, stream()))
    back = ref.gated_backward(dy, x, w, keep, "silu")
    for t, k in ((dx, "dx"), (dw, "dweight"), (db, "dbias")):
        assert_within(t, *back[k], k)
    assert frame_kept(xb, dx) and frame_kept(wb, dw)
    # without rows: zeros in dweight's columns alone
    a.rows = 0
    dw.fill_(3.0)
    ok(lbp, lbp.lib().vb_gated_linear_backward(ctypes.byref(a), None, 0, stream()))
    assert not dw.any() and not db.any() and frame_kept(wb, dw)
    assert es == dw.element_size()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n", [5, 300, 5000, 140001])
def test_norm_statistics_one_by_one(lbp, n, dtype):
    from linear_bound_propagation_amd import train
    rows = 6
    x = torch.randn(rows, n, device="cuda").to(dtype)
    y, mean, rstd = lbp.layer_norm(x, want_stats=True)
    for which in ("mean", "rstd"):
        out, buf = torch.empty_like(x), torch.full((rows + 2,), 7.0, device="cuda")
        a = train.vb_layer_norm_fwd(rows=rows, n=n, dtype=train.DTYPES[dtype], x=x.data_ptr(), ld_x=n, eps=1e-5,
                                    y=out.data_ptr(), ld_y=n, **{which: buf[1:].data_ptr()})
        ok(lbp, lbp.lib().vb_layer_norm_forward(ctypes.byref(a), stream()))
        assert torch.equal(out, y) and torch.equal(buf[1:-1], mean if which == "mean" else rstd)
        assert buf[0] == 7.0 and buf[-1] == 7.0


def test_calls_into_guarded_rows(lbp):
    """Rows of dx and y inside larger buffers, all lengths of a row's last chunk."""
    for dtype in TYPES:
        for n in list(range(1, 20)) + [127, 129, 1023, 1025, 4097]:
            rows = 3
            g = torch.Generator(device="cuda")
            g.manual_seed(n)
            x, dy, w = (torch.randn(*s, generator=g, device="cuda").to(dtype) for s in ((rows, n), (rows, n), (n,)))
            (yb, y), (db, dx), (ob, o) = framed(rows, n, dtype), framed(rows, n, dtype), framed(rows, n, dtype)
            lbp.layer_norm(x, w, out=y)
            _, mean, rstd = lbp.layer_norm(x, w, want_stats=True)
            assert_within(y, *ref.layer_norm(x, w, None, float(torch.tensor(1e-5)))["y"], f"y {n}")
            lbp.layer_norm_backward(dy, x, mean, rstd, w, dx=dx)
            assert_within(dx, *ref.layer_norm_backward(dy, x, mean, rstd, w, None)["dx"], f"dx {n}")
            lbp.dropout(x, 0.4, n, out=o)
            assert_within(o, *ref.dropout(x, 0.4, ref.kept(rows, n, 0.4, n, 0), None), f"dropout {n}")
            assert frame_kept(yb, y) and frame_kept(db, dx) and frame_kept(ob, o), (n, dtype)
