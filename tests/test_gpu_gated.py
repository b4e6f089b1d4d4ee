"""The gated linear layer and its backward pass against float64."""
import math

import pytest
import torch

import block_reference as ref
from helpers import ensure_built
from train_reference import assert_within

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
ACTS = ["none", "relu", "gelu", "silu"]
# (rows, n_in, n_out): a single token to large products, odd sizes, few and many of each
SIZES = [(1, 1, 1), (1, 100, 7), (2, 4096, 40), (1, 515, 2100), (4, 333, 1001), (3, 64, 5000), (7, 501, 399), (16, 128, 8192),
         (16, 1000, 33), (11, 9001, 33), (20, 9000, 130), (24, 300, 200), (32, 4100, 6500), (33, 17, 9), (64, 128, 64), (100, 784, 100), (129, 257, 130),
         (300, 64, 515), (1037, 201, 99), (512, 2048, 96), (130, 4096, 130)]


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def make(rows, n_in, n_out, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(dtype)

    return normal(rows, n_in), normal(2 * n_out, n_in, std=n_in ** -0.5), normal(2 * n_out, std=0.2), \
        normal(rows, n_out), normal(rows, 2 * n_out)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(lbp, size, dtype):
    x, w, b, _, _ = make(*size, dtype, 1)
    for name in ACTS:
        for bias in (b, None):
            what = f"gated {size} {dtype} {name} bias {bias is not None}"
            print(what, flush=True)
            y, pre = lbp.gated_linear(x, w, bias, act=name, want_pre=True)
            want = ref.gated(x, w, bias, name)
            assert_within(y, *want["y"], f"{what} y")
            assert_within(pre, *want["pre"], f"{what} pre")
            assert torch.equal(lbp.gated_linear(x, w, bias, act=name), y)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(lbp, size, dtype):
    x, w, _, dy, pre = make(*size, dtype, 2)
    for name in ACTS:
        for round_g in (False, True) if dtype != torch.float32 else (False,):
            what = f"gated backward {size} {dtype} {name} {round_g}"
            print(what, flush=True)
            got = lbp.gated_linear_backward(dy, x, w, pre, act=name, round_g=round_g)
            want = ref.gated_backward(dy, x, w, pre, name, round_g)
            for t, k in zip(got, ("dx", "dweight", "dbias")):
                assert_within(t, *want[k], f"{what} {k}")
    only = [lbp.gated_linear_backward(dy, x, w, pre, want_x=i == 0, want_weight=i == 1, want_bias=i == 2) for i in range(3)]
    both = lbp.gated_linear_backward(dy, x, w, pre)
    for i in range(3):
        assert torch.equal(only[i][i], both[i]), i
        assert all(only[i][j] is None for j in range(3) if j != i)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", [(2048, 512, 1024), (600, 1024, 2048), (4096, 256, 300)], ids=str)
def test_larger_products(lbp, size, dtype):
    """Tiles of every size, and parts of a reduction."""
    x, w, b, dy, pre = make(*size, dtype, 3)
    print(f"gated {size} {dtype}", flush=True)
    y, p = lbp.gated_linear(x, w, b, act="silu", want_pre=True)
    want = ref.gated(x, w, b, "silu")
    assert_within(y, *want["y"], "y")
    assert_within(p, *want["pre"], "pre")
    want = ref.gated_backward(dy, x, w, pre, "gelu")
    for t, k in zip(lbp.gated_linear_backward(dy, x, w, pre, act="gelu"), ("dx", "dweight", "dbias")):
        assert_within(t, *want[k], k)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", [(1, 700, 300), (3, 41, 2500), (9, 500, 77), (20, 1000, 51), (200, 130, 70), (520, 1100, 520)],
                         ids=str)
def test_strides_and_alignment(lbp, size, dtype):
    rows, n_in, n_out = size
    x, w, b, dy, pre = make(*size, dtype, 4)
    want = ref.gated(x, w, b, "gelu")
    back = ref.gated_backward(dy, x, w, pre, "silu")
    for pad, shift in ((8, 0), (5, 0), (3, 1), (1, 1)):
        def view(t):
            buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
            v = buf[:, shift:shift + t.shape[1]]
            v.copy_(t)
            return v

        print(f"gated strided {size} {dtype} {pad} {shift}", flush=True)
        buf = torch.full((rows, n_out + pad), 5.0, dtype=dtype, device="cuda")
        out = buf[:, shift:shift + n_out]
        y = lbp.gated_linear(view(x), view(w), b, act="gelu", out=out)
        assert y is out
        assert_within(y, *want["y"], "y")
        out.fill_(5.0)
        assert bool((buf == 5.0).all())
        got = lbp.gated_linear_backward(view(dy), view(x), view(w), view(pre))
        for t, k in zip(got, ("dx", "dweight", "dbias")):
            assert_within(t, *back[k], k)


@pytest.mark.parametrize("rows", [1, 3, 12, 40, 300])
def test_infinities_stay_in_their_rows_and_columns(lbp, rows):
    n_in, n_out = 130, 72
    for dtype in TYPES:
        x, w, b, dy, pre = make(rows, n_in, n_out, dtype, 5)
        clean = lbp.gated_linear(x, w, b)
        bad = x.clone()
        bad[rows - 1, 5] = math.nan
        y = lbp.gated_linear(bad, w, b)
        assert torch.isnan(y[rows - 1]).all() and torch.equal(y[:rows - 1], clean[:rows - 1])
        wb = w.clone()
        wb[n_out + 3, 7] = math.inf                     # up's row of output 3
        y = lbp.gated_linear(x, wb, b)
        ok = torch.ones(n_out, dtype=torch.bool, device="cuda")
        ok[3] = False
        assert not torch.isfinite(y[:, 3]).any() and torch.equal(y[:, ok], clean[:, ok])
        # a closed ReLU gate: no gradient, whatever the rest holds
        p = pre.clone()
        p[0, 4], p[0, n_out + 4] = -1.0, math.inf
        dx, dw, db = lbp.gated_linear_backward(dy, x, w, p, act="relu")
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()
        d = dy.clone()
        d[0, 4] = math.inf
        _, dw, db = lbp.gated_linear_backward(d, x, w, pre, act="silu", want_x=False)
        at = torch.zeros(2 * n_out, dtype=torch.bool, device="cuda")
        at[4] = at[n_out + 4] = True
        ref_dw = lbp.gated_linear_backward(dy, x, w, pre, act="silu")[1]
        assert not torch.isfinite(dw[at]).any() and torch.equal(dw[~at], ref_dw[~at])
        assert not torch.isfinite(db[at]).any() and torch.isfinite(db[~at]).all()


def test_no_rows(lbp):
    w = torch.randn(40, 30, device="cuda")
    x = torch.empty(0, 30, device="cuda")
    y, pre = lbp.gated_linear(x, w, want_pre=True)
    assert y.shape == (0, 20) and pre.shape == (0, 40)
    dx, dw, db = lbp.gated_linear_backward(y, x, w, pre)
    assert dx.shape == (0, 30) and dw.shape == (40, 30) and not dw.any() and not db.any()


def test_workspaces_are_enough(lbp):
    """A workspace made for the sizes serves every activation, with and without pre."""
    for dtype in TYPES:
        for size in ((5, 300, 70), (300, 1100, 77), (64, 8192, 64)):
            x, w, b, dy, pre = make(*size, dtype, 7)
            ws, wb = lbp.gated_linear_workspace(x, w), lbp.gated_linear_workspace(x, w, backward=True)
            for name in ACTS:
                y = lbp.gated_linear(x, w, b, act=name, ws=ws)
                assert torch.equal(y, lbp.gated_linear(x, w, b, act=name))
                for round_g in (False, True):
                    for want in ((True, True, True), (True, False, False), (False, True, True)):
                        lbp.gated_linear_backward(dy, x, w, pre, name, *want, ws=wb, round_g=round_g)
    torch.cuda.synchronize()


def test_gradient_against_differences(lbp):
    """Central differences of the float64 formula, h = 1e-4: error h^2 / 6 of third derivatives
    below 1000 (2e-6) and 1e-10 of rounding."""
    x, w, b, dy, _ = make(9, 21, 13, torch.float32, 9)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    h = 1e-4
    for name in ("none", "gelu", "silu"):
        pre = lbp.gated_linear(x, w, b, act=name, want_pre=True)[1]
        grads = lbp.gated_linear_backward(dy, x, w, pre, act=name)
        bounds = ref.gated_backward(dy, x, w, pre, name)

        def f(x, w, b):
            v = ref.mm(x, w.t()) + b
            return (ref.act(v[:, :13], name) * v[:, 13:] * dy.double()).sum()

        at = [x.double(), w.double(), b.double()]
        for i, k in enumerate(("dx", "dweight", "dbias")):
            v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
            hi, lo = list(at), list(at)
            hi[i], lo[i] = at[i] + h * v, at[i] - h * v
            slope = float((f(*hi) - f(*lo)) / (2 * h))
            # pre is a float32 number: 30 units of rounding of sums of 22 products below 10
            allowed = float((bounds[k][1] * v.abs()).sum()) + 1e-4 * float(v.abs().mean()) * at[i].numel() ** 0.5
            assert abs(float((grads[i].double() * v).sum()) - slope) <= allowed, (name, k)


def test_graph(lbp):
    x, w, b, dy, _ = make(300, 256, 200, torch.bfloat16, 10)
    ws, wb = lbp.gated_linear_workspace(x, w), lbp.gated_linear_workspace(x, w, backward=True)

    def run():
        y, pre = lbp.gated_linear(x, w, b, want_pre=True, ws=ws)
        return (y, pre) + lbp.gated_linear_backward(dy, x, w, pre, ws=wb)

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = run()
    for k in range(3):
        x.copy_(make(300, 256, 200, torch.bfloat16, 30 + k)[0])
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(kept, eager)), k
