"""Softmax cross entropy and its gradient against float64."""
import math

import pytest
import torch

import train_reference as ref
from helpers import ensure_built

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
SIZES = [(1, 1), (1, 2), (16, 10), (5, 64), (7, 99), (33, 257), (3, 1000), (130, 100), (9, 4096), (2, 32768),
         (3, 50001), (2, 100003), (1, 262144), (700, 31)]


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def make(rows, classes, dtype, seed, std=3.0, ignored=0.2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = (torch.randn(rows, classes, generator=g, device="cuda") * std).to(dtype)
    y = torch.randint(0, classes, (rows,), generator=g, device="cuda")
    drop = torch.rand(rows, generator=g, device="cuda") < ignored
    return z, torch.where(drop, torch.full_like(y, -100), y)


def check(lbp, z, y, eps, scale, what, ignore=-100, **kw):
    loss, row, grad = lbp.cross_entropy(z, y, ignore_index=ignore, label_smoothing=eps, grad_scale=scale, **kw)
    zz = z if kw.get("keep") is None else kw["keep"]
    wl, wr, wg = ref.cross_entropy(zz, y, ignore, eps, scale)
    classes, dt = z.shape[1], z.dtype
    # exp: 2^-18 relative for 16-bit logits (2^-20 for float32, with its argument's rounding);
    # the sum adds classes 2^-24 at worst; the loss is a difference of logits beside it
    e = ref.ACT[dt] + (classes + 8) * ref.U32
    top = z.double().cpu().nan_to_num(0, 0, 0).abs().amax(1) + math.log(classes) + 1
    er = e + 8 * ref.U32 * top * (1 + (classes * eps if eps else 0))
    used = (y.cpu() != ignore)
    ref.assert_within(row, wr, torch.where(used, er, torch.zeros_like(er)), f"{what} row_loss")
    n = max(int(used.sum()), 1)
    ref.assert_within(loss, wl.reshape(1), float(er[used].sum() / n + 4 * ref.U32 * wr.abs().nan_to_num(0, 0, 0).max())
                      if used.any() else 0.0, f"{what} loss")
    # p (2 e relative), minus two constants, times the scale
    s = abs(scale) / n
    p = torch.softmax(z.double().cpu(), 1).nan_to_num(0, 0, 0)
    eg = s * (2 * e * p + 4 * ref.U32 * (p + 1.0 / classes) + 4 * ref.U32 * (wg.nan_to_num(0, 0, 0).abs() / max(s, 1e-300) > 0.5))
    eg = eg + ref.UNIT[dt] * (wg.nan_to_num(0, 0, 0).abs() + eg) + ref.TINY[dt] + 4 * ref.U32 * s * p
    ref.assert_within(grad, wg, eg, f"{what} dlogits")
    return loss, row, grad


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_loss_and_gradient(lbp, size, dtype):
    for i, (eps, scale) in enumerate(((0.0, 1.0), (0.1, 1.0), (0.0, 1024.0), (1.0, -2.0))):
        z, y = make(*size, dtype, seed=i)
        what = f"loss {size} {dtype} smoothing {eps} scale {scale}"
        print(what, flush=True)
        check(lbp, z, y, eps, scale, what)
        loss, row, none = lbp.cross_entropy(z, y, label_smoothing=eps, grad_scale=scale, want_grad=False)
        full = lbp.cross_entropy(z, y, label_smoothing=eps, grad_scale=scale)
        assert none is None and torch.equal(loss, full[0]) and torch.equal(row, full[1])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("classes", [10, 100, 4100, 50001, 200000])
def test_masked_classes_and_odd_rows(lbp, classes, dtype):
    """-inf logits, a label on a masked class, labels out of range, a NaN, +inf, a row without any
    class, the lowest finite value, ignored rows: each stays in its row."""
    z, y = make(14, classes, dtype, seed=4, ignored=0.0)
    low = torch.finfo(dtype).min
    z[1, ::2] = float("-inf")
    y[1] = 1
    z[2, 5] = float("-inf")
    y[2] = 5                            # loss +inf, gradient finite
    y[3] = classes                      # out of range
    y[4] = -1
    z[5, 3] = float("nan")
    z[6, 7] = float("inf")
    z[7] = float("-inf")
    z[8] = low
    z[9, 1:] = low
    y[9] = 0
    y[10] = -100
    z[10] = float("nan")                # ignored: not looked at
    z[11] = torch.finfo(dtype).max / 2
    z[12, 1:] = float("-inf")
    y[12] = 0                           # one class left: loss 0
    print(f"odd rows {classes} {dtype}", flush=True)
    loss, row, grad = check(lbp, z, y, 0.0, 3.0, f"odd rows {classes} {dtype}")
    assert torch.isnan(loss).all()
    assert row[2] == math.inf and torch.isfinite(grad[2]).all()
    for r in (3, 4, 5, 6, 7):
        assert torch.isnan(row[r]) and torch.isnan(grad[r]).any()
    assert row[10] == 0 and (grad[10] == 0).all()
    assert row[12] == 0 and (grad[12] == 0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("pad, shift", [(8, 0), (5, 0), (3, 1)], ids=str)
@pytest.mark.parametrize("classes", [10, 1001, 40004, 130001])
def test_strides_and_in_place(lbp, classes, pad, shift, dtype):
    z, y = make(6, classes, dtype, seed=9)
    buf = torch.full((6, classes + pad), float("nan"), dtype=dtype, device="cuda")
    view = buf[:, shift:shift + classes]
    view.copy_(z)
    print(f"strided {classes} {pad} {shift} {dtype}", flush=True)
    want = lbp.cross_entropy(z, y, label_smoothing=0.1)
    got = check(lbp, view, y, 0.1, 1.0, "strided")
    out = torch.full_like(buf, 5.0)
    ov = out[:, shift:shift + classes]
    lbp.cross_entropy(view, y, label_smoothing=0.1, dlogits=ov)
    assert torch.equal(ov, got[2])
    outside = torch.ones(classes + pad, dtype=torch.bool, device="cuda")
    outside[shift:shift + classes] = False
    assert (out[:, outside] == 5.0).all()
    loss, row, grad = lbp.cross_entropy(view, y, label_smoothing=0.1, dlogits=view)     # over the logits
    assert grad is view and torch.equal(view, got[2]) and torch.equal(row, got[1]) and torch.equal(loss, got[0])
    assert torch.isnan(buf[:, outside]).all()
    assert want[1].shape == row.shape


def test_every_row_ignored_and_no_rows(lbp):
    for dtype in TYPES:
        z, y = make(5, 33, dtype, seed=2)
        loss, row, grad = lbp.cross_entropy(z, torch.full_like(y, 7), ignore_index=7)
        assert loss == 0 and (row == 0).all() and (grad == 0).all()
        loss, row, grad = lbp.cross_entropy(z[:0], y[:0])
        assert loss == 0 and row.shape == (0,) and grad.shape == (0, 33)
        # an ignore_index inside the classes is ignored too
        y = torch.arange(5, device="cuda")
        loss, row, grad = lbp.cross_entropy(z, y, ignore_index=2)
        assert row[2] == 0 and (grad[2] == 0).all() and (row[[0, 1, 3, 4]] > 0).all()


def test_gradient_against_differences(lbp):
    """Central differences of the library's loss; allowed: truncation (from float64) and rounding."""
    z, y = make(12, 40, torch.float32, seed=14, std=1.5)
    h = 2.0 ** -6
    for eps in (0.0, 0.2):
        grad = lbp.cross_entropy(z, y, label_smoothing=eps)[2]
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        d = torch.randn(z.shape, generator=g, device="cuda")
        zp, zm = z + h * d, z - h * d
        d = ((zp.double() - zm.double()) / (2 * h)).cpu()
        fd = float((lbp.cross_entropy(zp, y, label_smoothing=eps)[0].double()
                    - lbp.cross_entropy(zm, y, label_smoothing=eps)[0].double()) / (2 * h))
        fd64 = float((ref.cross_entropy(zp, y, -100, eps, 1.0)[0] - ref.cross_entropy(zm, y, -100, eps, 1.0)[0]) / (2 * h))
        slope64 = float((ref.cross_entropy(z, y, -100, eps, 1.0)[2] * d).sum())
        slope = float((grad.double().cpu() * d).sum())
        rounding = 2.0 ** -18 * 8 / h
        assert abs(fd - slope) <= abs(fd64 - slope64) + rounding, (fd, slope)
        assert abs(fd64 - slope64) < 1e-3


def test_stream_graph_and_repeats(lbp):
    z, y = make(65, 3001, torch.bfloat16, seed=21)
    ws = lbp.cross_entropy_workspace(z)
    ws.fill_(255)
    first = lbp.cross_entropy(z, y, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = lbp.cross_entropy(z, y, ws=ws)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = lbp.cross_entropy(z, y, ws=ws)
    for i in range(3):
        z.copy_(make(65, 3001, torch.bfloat16, seed=30 + i)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, lbp.cross_entropy(z, y))), i


def test_refusals_of_the_binding(lbp):
    z, y = make(6, 9, torch.float32, seed=1)
    for call, text in (
            (lambda: lbp.cross_entropy(z[0], y), "matrix"), (lambda: lbp.cross_entropy(z.t(), y), "contiguous"),
            (lambda: lbp.cross_entropy(z, y.int()), "labels"), (lambda: lbp.cross_entropy(z, y[:5]), "labels"),
            (lambda: lbp.cross_entropy(z, y.cpu()), "labels"), (lambda: lbp.cross_entropy(z.double(), y), "float32"),
            (lambda: lbp.cross_entropy(z, y, dlogits=z[:, :8]), "dlogits"),
            (lambda: lbp.cross_entropy(z, y, dlogits=z.half()), "dlogits")):
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(lbp.VBError, match="label_smoothing"):
        lbp.cross_entropy(z, y, label_smoothing=2.0)
