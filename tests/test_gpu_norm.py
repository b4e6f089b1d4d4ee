"""Layer norm and its backward pass against float64."""
import math

import pytest
import torch

import block_reference as ref
from helpers import ensure_built
from train_reference import U32, assert_within

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# a wavefront a row, several, a workgroup, the longest in registers, longer ones; odd ends of each
SIZES = [(1, 1), (5, 1), (1, 2), (16, 100), (3, 255), (7, 513), (130, 1001), (600, 64), (33, 2001), (9, 2048), (5, 4095),
         (6, 8192), (3, 8200), (2, 16384), (3, 16387), (2, 40000), (1, 65536), (2, 70001), (1, 200003)]


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def make(rows, n, dtype, seed, mean=0.3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    return ((normal(rows, n) + mean) * 1.7).to(dtype), (1 + 0.2 * normal(n)).to(dtype), (0.3 * normal(n)).to(dtype), \
        normal(rows, n).to(dtype), normal(rows, n).to(dtype)


def check(got, want, what):
    for name, t in got.items():
        assert_within(t, *want[name], f"{what} {name}")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(lbp, size, dtype):
    x, w, b, _, _ = make(*size, dtype, 1)
    for k, (wk, bk) in enumerate(((w, b), (None, None), (w, None), (None, b))):
        print(f"norm {size} {dtype} {k}", flush=True)
        y, mean, rstd = lbp.layer_norm(x, wk, bk, eps=1e-5, want_stats=True)
        check({"y": y, "mean": mean, "rstd": rstd}, ref.layer_norm(x, wk, bk, float(torch.tensor(1e-5))), f"norm {size} {dtype} {k}")
        assert torch.equal(lbp.layer_norm(x, wk, bk), y)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(lbp, size, dtype):
    x, w, b, dy, res = make(*size, dtype, 2)
    _, mean, rstd = lbp.layer_norm(x, w, b, want_stats=True)
    for k, (wk, rk) in enumerate(((w, None), (w, res), (None, res))):
        what = f"norm backward {size} {dtype} {k}"
        print(what, flush=True)
        dx, dw, db = lbp.layer_norm_backward(dy, x, mean, rstd, wk, dresidual=rk)
        check({"dx": dx, "dweight": dw, "dbias": db}, ref.layer_norm_backward(dy, x, mean, rstd, wk, rk), what)
    # each gradient alone, with the same bits
    only = [lbp.layer_norm_backward(dy, x, mean, rstd, w, dresidual=res, want_x=i == 0, want_weight=i == 1, want_bias=i == 2)
            for i in range(3)]
    both = lbp.layer_norm_backward(dy, x, mean, rstd, w, dresidual=res)
    for i in range(3):
        assert torch.equal(only[i][i], both[i]), i
        assert all(only[i][j] is None for j in range(3) if j != i)


@pytest.mark.parametrize("size", [(2000, 256), (5000, 100), (1300, 4096), (700, 9000), (300, 40000)], ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_many_rows(lbp, size, dtype):
    """More rows than workgroups that keep sums."""
    x, w, b, dy, res = make(*size, dtype, 3)
    print(f"norm {size} {dtype}", flush=True)
    y, mean, rstd = lbp.layer_norm(x, w, b, want_stats=True)
    check({"y": y, "mean": mean, "rstd": rstd}, ref.layer_norm(x, w, b, float(torch.tensor(1e-5))), f"norm {size} {dtype}")
    dx, dw, db = lbp.layer_norm_backward(dy, x, mean, rstd, w, dresidual=res)
    check({"dx": dx, "dweight": dw, "dbias": db}, ref.layer_norm_backward(dy, x, mean, rstd, w, res), f"backward {size} {dtype}")


@pytest.mark.parametrize("mean", [100.0, 3000.0, -1e6])
def test_rows_far_off_zero(lbp, mean):
    """The variance of float32 rows comes from differences: 1e6 +- 1 keeps what its numbers hold."""
    for n in (100, 5000, 70000):
        x, w, b, _, _ = make(4, n, torch.float32, 5, mean=mean)
        y, m, r = lbp.layer_norm(x, w, b, want_stats=True)
        check({"y": y, "mean": m, "rstd": r}, ref.layer_norm(x, w, b, float(torch.tensor(1e-5))), f"far off {mean} {n}")


@pytest.mark.parametrize("n", [100, 4096, 9001, 140001])
def test_one_large_element(lbp, n):
    """An element a million times the others, the first one or another: the others keep the bits that
    their own size gives them (bounds of differences from the mean, not from the large one)."""
    for at in (0, n // 2, n - 1):
        x, w, b, _, _ = make(3, n, torch.float32, 6)
        x[:, at] = torch.tensor([1e6, -3e5, 1e3], device="cuda")
        y, m, r = lbp.layer_norm(x, w, b, want_stats=True)
        check({"y": y, "mean": m, "rstd": r}, ref.layer_norm(x, w, b, float(torch.tensor(1e-5))), f"large {n} {at}")


def test_an_infinite_weight_at_the_end(lbp):
    """Elements that a row's last chunk shares with the one before it count once."""
    for n in (13, 1003, 5001):
        x, w, b, dy, _ = make(5, n, torch.bfloat16, 7)
        _, mean, rstd = lbp.layer_norm(x, w, b, want_stats=True)
        w[n - 3] = math.inf
        dy[:, n - 3] = 1.0
        x[:, n - 3] = x.amax() + 1
        dx, dw, db = lbp.layer_norm_backward(dy, x, mean, rstd, w)
        want = ref.layer_norm_backward(dy, x, mean, rstd, w, None)
        assert torch.equal(torch.isnan(dx), torch.isnan(want["dx"][0])), n
        assert_within(dw, *want["dweight"], f"dweight {n}")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n", [7, 300, 3001, 9001, 140001])
def test_strides_alignment_and_in_place(lbp, n, dtype):
    rows = 5
    x, w, b, dy, res = make(rows, n, dtype, 6)
    y, mean, rstd = lbp.layer_norm(x, w, b, want_stats=True)
    dx, dw, db = lbp.layer_norm_backward(dy, x, mean, rstd, w, dresidual=res)
    for pad, shift in ((8, 0), (5, 0), (3, 1)):
        def view(t):
            buf = torch.full((rows, n + pad), 9.0, dtype=dtype, device="cuda")
            buf[:, shift:shift + n] = t
            return buf, buf[:, shift:shift + n]

        def untouched(buf):
            edge = buf.clone()
            edge[:, shift:shift + n] = 9.0
            return bool((edge == 9.0).all())

        print(f"strided {n} {dtype} {pad} {shift}", flush=True)
        (_, xv), (_, dyv), (_, rv) = view(x), view(dy), view(res)
        ob, ov = view(torch.zeros_like(x))
        assert lbp.layer_norm(xv, w, b, out=ov) is ov and torch.equal(ov, y) and untouched(ob)
        got = lbp.layer_norm_backward(dyv, xv, mean, rstd, w, dresidual=rv, dx=ov)
        assert got[0] is ov and untouched(ob)
        assert all(torch.equal(a, c) for a, c in zip(got, (dx, dw, db)))
        for k in (0, 1):                                    # over dy, over dresidual
            (b0, v0), (b1, v1) = view(dy), view(res)
            got = lbp.layer_norm_backward(v0, xv, mean, rstd, w, dresidual=v1, dx=(v0, v1)[k])
            assert all(torch.equal(a, c) for a, c in zip(got, (dx, dw, db))) and untouched(b0) and untouched(b1)
        xb, xv = view(x)
        assert torch.equal(lbp.layer_norm(xv, w, b, out=xv), y) and untouched(xb)
    # one row: any stride
    one = lbp.layer_norm(x[:1].as_strided((1, n), (1, 1)), w, b)
    assert torch.equal(one, y[:1])


def test_infinities_and_equal_numbers(lbp):
    for n in (40, 3000, 90000):
        x, w, b, dy, _ = make(6, n, torch.float32, 8)
        x[1, 3] = math.inf
        x[2, n - 1] = math.nan
        x[3] = 5.0
        x[4] = torch.finfo(torch.float32).max / 2
        y, mean, rstd = lbp.layer_norm(x, w, b, want_stats=True)
        assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
        assert torch.equal(y[3], b) and float(mean[3]) == 5.0
        assert torch.equal(y[4], b) and float(mean[4]) == torch.finfo(torch.float32).max / 2
        clean = torch.tensor([0, 5], device="cuda")
        want = lbp.layer_norm(x[clean].contiguous(), w, b)
        assert torch.equal(y[clean], want)
        assert torch.isnan(lbp.layer_norm(x, w, b, eps=0.0)[3]).all()
        # a bad row spoils dweight, not the other rows' dx
        dx, dw, db = lbp.layer_norm_backward(dy, x, mean, rstd, w)
        good = lbp.layer_norm_backward(dy[clean].contiguous(), x[clean].contiguous(), mean[clean], rstd[clean], w)
        assert torch.equal(dx[clean], good[0]) and torch.isnan(dw).all() and torch.isfinite(db).all()
        assert torch.isnan(dx[1]).all() and torch.isnan(dx[2]).all()


def test_no_rows(lbp):
    x = torch.empty(0, 50, device="cuda")
    w = torch.ones(50, device="cuda")
    y, mean, rstd = lbp.layer_norm(x, w, w, want_stats=True)
    assert y.shape == (0, 50) and mean.shape == rstd.shape == (0,)
    dx, dw, db = lbp.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, 50) and not dw.any() and not db.any()
    assert lbp.layer_norm_backward(x, x, mean, rstd, w, want_weight=False, want_bias=False)[0].shape == (0, 50)


def test_gradient_against_differences(lbp):
    """<dx, v> and <dw, u> against central differences of the float64 formula, whose own error
    is h^2 / 6 of a third derivative (here below 100): 2e-7 with h = 1e-4."""
    x, w, b, dy, res = make(7, 33, torch.float32, 11)
    _, mean, rstd = lbp.layer_norm(x, w, b, want_stats=True)
    dx, dw, db = lbp.layer_norm_backward(dy, x, mean, rstd, w, dresidual=res)

    def f(x, w, b):
        c = x - x.mean(1, keepdim=True)
        y = c * ((c * c).mean(1, keepdim=True) + 1e-5) ** -0.5 * w + b
        return (y * dy.double()).sum() + (x * res.double()).sum()

    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    h = 1e-4
    at = [x.double(), w.double(), b.double()]
    bounds = ref.layer_norm_backward(dy, x, mean, rstd, w, res)
    for i, (grad, name) in enumerate(((dx, "dx"), (dw, "dweight"), (db, "dbias"))):
        v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + h * v, at[i] - h * v
        slope = float((f(*hi) - f(*lo)) / (2 * h))
        # the gradient's own bound, that of the float32 statistics it is given (a few units of
        # n u each), and the difference's error
        allowed = float((bounds[name][1] * v.abs()).sum()) + 40 * 33 * U32 * float((grad.double() * v).abs().sum() + v.abs().sum()) + 2e-5
        assert abs(float((grad.double() * v).sum()) - slope) <= allowed, name


def test_streams_and_graph(lbp):
    """On another stream, and captured and replayed with new inputs between eager calls."""
    x, w, b, dy, res = make(300, 1000, torch.bfloat16, 13)
    ws = lbp.layer_norm_workspace(x)

    def run():
        y, mean, rstd = lbp.layer_norm(x, w, b, want_stats=True)
        return (y, mean, rstd) + lbp.layer_norm_backward(dy, x, mean, rstd, w, dresidual=res, ws=ws)

    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    for k in range(3):
        x.copy_(make(300, 1000, torch.bfloat16, 20 + k)[0])
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(kept, eager)), k
