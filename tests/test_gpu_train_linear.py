"""The fused linear layer and its backward pass against float64."""
import pytest
import torch

import train_reference as ref
from helpers import ensure_built

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
ACTS = ["none", "relu", "gelu", "silu"]
# (rows, n_in, n_out): single tokens, sizes that divide by nothing, tile edges, long reductions
SIZES = [(1, 1, 1), (1, 64, 64), (2, 8, 3), (3, 5, 7), (1, 4096, 300), (16, 784, 100), (16, 100, 10), (17, 33, 65),
         (33, 31, 1), (64, 64, 64), (65, 100, 129), (128, 256, 512), (5, 8191, 50), (300, 1000, 130),
         (257, 72, 511), (1024, 512, 384), (640, 2056, 264), (2, 1001, 4097)]


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def case(rows, n_in, n_out, dtype, seed=0):
    g = gen(seed)
    return (normal(g, rows, n_in, dtype=dtype), normal(g, n_out, n_in, std=n_in ** -0.5, dtype=dtype),
            normal(g, n_out, std=0.1, dtype=dtype), normal(g, rows, n_out, dtype=dtype))


def check_forward(lbp, x, w, b, r, act, what, **kw):
    got, pre = lbp.linear(x, w, b, r, act=act, want_pre=True, **kw)
    y, v, ey, ev = ref.linear(x, w, b, r, act)
    ref.assert_within(got, y, ey, f"{what} y")
    ref.assert_within(pre, v, ev, f"{what} pre")
    return got, pre


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(lbp, size, dtype):
    for i, act in enumerate(ACTS):
        x, w, b, r = case(*size, dtype, seed=i)
        what = f"linear {size} {dtype} {act}"
        print(what, flush=True)
        check_forward(lbp, x, w, b if i != 1 else None, r if i % 2 else None, act, what)
        # without pre: the same y
        y = lbp.linear(x, w, b, None, act=act)
        assert torch.equal(y, lbp.linear(x, w, b, None, act=act, want_pre=True)[0]), what


def check_backward(lbp, dy, x, w, saved, act, what, **kw):
    out = lbp.linear_backward(dy, x, w, act=act, saved=saved, want_residual=True, **kw)
    want = ref.linear_backward(dy, x, w, saved, act)
    for name, t in zip(("dx", "dweight", "dbias", "dresidual"), out):
        ref.assert_within(t, *want[name], f"{what} {name}")
    return out


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(lbp, size, dtype):
    rows, n_in, n_out = size
    for i, act in enumerate(ACTS):
        x, w, b, r = case(*size, dtype, seed=10 + i)
        dy = normal(gen(20 + i), rows, n_out, dtype=dtype)
        saved = {"none": None, "relu": r.clamp_min(0)}.get(act, r)
        what = f"linear_backward {size} {dtype} {act}"
        print(what, flush=True)
        out = check_backward(lbp, dy, x, w, saved, act, what)
        # each gradient alone is the same
        for k, name in enumerate(("want_x", "want_weight", "want_bias", "want_residual")):
            flags = dict(want_x=False, want_weight=False, want_bias=False, want_residual=False)
            flags[name] = True
            one = lbp.linear_backward(dy, x, w, act=act, saved=saved, **flags)
            assert torch.equal(one[k], out[k]), (what, name)
            assert all(t is None for j, t in enumerate(one) if j != k)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("pad, shift", [(8, 0), (5, 0), (16, 8), (3, 1)], ids=str)
@pytest.mark.parametrize("size", [(1, 96, 40), (12, 301, 77), (37, 120, 72), (200, 250, 136), (300, 515, 129)], ids=str)
def test_strides_and_alignment(lbp, size, pad, shift, dtype):
    """Operands and outputs inside wider buffers, from an odd element on; nothing outside is written."""
    rows, n_in, n_out = size
    print(f"strides {size} pad {pad} shift {shift} {dtype}", flush=True)

    def inside(t, around=float("nan")):
        buf = torch.full((t.shape[0], t.shape[1] + pad), around, dtype=dtype, device="cuda")
        view = buf[:, shift:shift + t.shape[1]]
        view.copy_(t)
        return buf, view

    x, w, b, r = case(*size, dtype, seed=3)
    (_, xv), (_, wv), (_, rv) = inside(x), inside(w), inside(r)
    ybuf, yv = inside(torch.zeros_like(r), 7.0)
    check_forward(lbp, xv, wv, b, rv, "silu", "strided", out=yv)
    outside = torch.ones(n_out + pad, dtype=torch.bool, device="cuda")
    outside[shift:shift + n_out] = False
    assert (ybuf[:, outside] == 7.0).all()
    dy = normal(gen(5), rows, n_out, dtype=dtype)
    _, dyv = inside(dy)
    check_backward(lbp, dyv, xv, wv, rv, "gelu", "strided")
    check_backward(lbp, dyv, xv, wv, None, "none", "strided")
    # y over the residual
    alias = rv.clone()
    buf, av = inside(alias, 7.0)
    y = lbp.linear(xv, wv, b, av, act="relu", out=av)
    assert y is av and torch.equal(y, lbp.linear(xv, wv, b, rv, act="relu"))
    assert (buf[:, outside] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [1, 9, 130])
def test_infinities_and_nan_stay_in_their_rows_and_columns(lbp, rows, dtype):
    n_in, n_out = 200, 136
    x, w, b, r = case(rows, n_in, n_out, dtype, seed=6)
    clean = lbp.linear(x, w, b, r)
    x[rows // 2, 17] = float("nan")
    w[3, 199] = float("inf")
    print(f"nan / inf rows {rows} {dtype}", flush=True)
    got = lbp.linear(x, w, b, r)
    want = ref.linear(x, w, b, r, "none")[0]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.isnan(got[rows // 2]).all()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[rows // 2] = False
    rest[:, 3] = False
    assert torch.equal(got[rest], clean[rest])
    col = torch.arange(rows, device="cuda") != rows // 2
    assert torch.isinf(got[col, 3]).all() and torch.equal(got[col, 3].double(), want[col, 3])
    # a ReLU passes NaN on; its gradient is zero wherever the saved output is not positive
    assert torch.isnan(lbp.linear(x, w, b, r, act="relu")[rows // 2]).all()
    dy = torch.full((rows, n_out), float("nan"), dtype=dtype, device="cuda")
    dx, dw, db, dr = lbp.linear_backward(dy, clean.new_zeros(rows, n_in), clean.new_ones(n_out, n_in), act="relu",
                                         saved=torch.zeros_like(clean), want_residual=True)
    for t in (dx, dw, db, dr):
        assert (t == 0).all()


def test_large_and_small_float32_values(lbp):
    """Float32 operands over the whole exponent range keep float32 accuracy."""
    rows, n_in, n_out = 150, 256, 200
    x, w, b, r = case(rows, n_in, n_out, F32, seed=8)
    for sx, sw in ((1e30, 1e-30), (1e-20, 1e-10), (3e38, 1e-3), (1e-30, 1.0), (1e18, 1e18)):
        xs = (x.clamp(-1, 1) * sx)
        ws = (w.clamp(-1, 1) * sw)
        print(f"scales {sx} {sw}", flush=True)
        got = lbp.linear(xs, ws)
        want, _, e, _ = ref.linear(xs, ws, None, None, "none")
        ref.assert_within(got, want, e + n_in * 2.0 ** -126 * float(max(sx * 2.0 ** -8, sw * 2.0 ** -8, 1.0)), "scales")


def test_no_rows(lbp):
    for dtype in TYPES:
        x, w, b, r = case(4, 12, 10, dtype)
        y, pre = lbp.linear(x[:0], w, b, r[:0], act="gelu", want_pre=True)
        assert y.shape == (0, 10) and pre.shape == (0, 10)
        dx, dw, db, dr = lbp.linear_backward(r[:0], x[:0], w, act="gelu", saved=r[:0], want_residual=True)
        assert dx.shape == (0, 12) and dr.shape == (0, 10)
        assert dw.shape == (10, 12) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(lbp, act):
    """Directional derivatives of sum(y * dy) by central differences of the library's own
    forward pass, against the library's gradients.  Allowed: the difference's own truncation
    (taken from float64) and the float32 rounding of the two forward passes."""
    rows, n_in, n_out, h = 40, 70, 50, 2.0 ** -7
    x, w, b, r = case(rows, n_in, n_out, F32, seed=31)
    dy = normal(gen(32), rows, n_out)
    y, pre = lbp.linear(x, w, b, r, act=act, want_pre=True)
    if act == "relu":       # stay off the kink: no pre-activation changes sign under the steps
        r = torch.where(pre.abs() < 0.5, r + torch.where(pre >= 0, 1.0, -1.0), r)
        y, pre = lbp.linear(x, w, b, r, act=act, want_pre=True)
    saved = {"none": None, "relu": y}.get(act, pre)
    grads = lbp.linear_backward(dy, x, w, act=act, saved=saved, want_residual=True)
    g = gen(33)
    for k, name in enumerate(("x", "weight", "bias", "residual")):
        args = [x, w, b, r]
        d = normal(g, *args[k].shape, std=0.05 if name == "weight" else 0.2)
        plus, minus = list(args), list(args)
        plus[k], minus[k] = args[k] + h * d, args[k] - h * d
        d = (plus[k].double() - minus[k].double()) / (2 * h)    # the step as rounded
        lib = [(lbp.linear(*a, act=act).double() * dy.double()).sum() for a in (plus, minus)]
        exact, e = zip(*[ref.linear(*a, act)[0::2] for a in (plus, minus)])
        fd = (lib[0] - lib[1]) / (2 * h)
        fd64 = ((exact[0] - exact[1]) * dy.double()).sum() / (2 * h)
        want = ref.linear_backward(dy, x, w, saved, act)[("dx", "dweight", "dbias", "dresidual")[k]]
        slope64 = (want[0] * d).sum()
        slope = (grads[k].double() * d).sum()
        allowed = (fd64 - slope64).abs() + ((e[0] + e[1]) * dy.double().abs()).sum() / (2 * h) \
            + (want[1] * d.abs()).sum()
        assert (fd - slope).abs() <= allowed, (name, float(fd), float(slope), float(allowed))
        assert (fd64 - slope64).abs() <= 1e-3 * (1 + slope64.abs()), name


def test_other_stream_and_repeated_calls(lbp):
    """On a stream of the caller's, with a kept workspace: bitwise the same each time."""
    x, w, b, r = case(200, 520, 264, BF16, seed=40)
    dy = normal(gen(41), 200, 264, dtype=BF16)
    y0 = lbp.linear(x, w, b, r, act="silu")
    g0 = lbp.linear_backward(dy, x, w, act="silu", saved=r, want_residual=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = lbp.linear_workspace(x, w, backward=True)
        ws.fill_(255)
        for _ in range(3):
            assert torch.equal(lbp.linear(x, w, b, r, act="silu", ws=ws), y0)
            g = lbp.linear_backward(dy, x, w, act="silu", saved=r, want_residual=True, ws=ws)
            assert all(torch.equal(a, c) for a, c in zip(g, g0))
    s.synchronize()


@pytest.mark.parametrize("size, dtype", [((4, 600, 300), BF16), ((96, 300, 200), F32), ((520, 512, 512), F16)], ids=str)
def test_captured_in_a_graph(lbp, size, dtype):
    rows, n_in, n_out = size
    x, w, b, r = case(*size, dtype, seed=50)
    dy = normal(gen(51), rows, n_out, dtype=dtype)
    wf, wb = lbp.linear_workspace(x, w), lbp.linear_workspace(x, w, backward=True)

    def step():
        y, pre = lbp.linear(x, w, b, r, act="gelu", want_pre=True, ws=wf)
        return (y, pre) + lbp.linear_backward(dy, x, w, act="gelu", saved=pre, want_residual=True, ws=wb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        x.copy_(normal(gen(60 + i), rows, n_in, dtype=dtype))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(outs, step()):
            assert torch.equal(a, c), i


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 16, 17, 32, 33])
def test_few_rows_at_every_alignment(lbp, rows, dtype):
    """Weight rows at every distance from a 16-byte boundary, widths about a whole number of chunks
    and runs, more and fewer weight rows than a period."""
    for n_in in (1, 3, 7, 8, 9, 63, 130, 1031, 2303):
        for n_out in (1, 3, 40, 129, 2100):
            for shift in (0, 1, 3):
                if n_out == 2100 and (n_in > 200 or shift):
                    continue
                x, w, b, r = case(rows, n_in, n_out, dtype, seed=n_in + n_out)
                buf = torch.full((n_out * n_in + 16,), float("nan"), dtype=dtype, device="cuda")
                wv = buf[shift:shift + n_out * n_in].view(n_out, n_in)
                wv.copy_(w)
                check_forward(lbp, x, wv, b, r, "none", f"few rows {rows} {n_in} {n_out} {shift} {dtype}")
    # workgroups of 64 weight rows
    for n_in, n_out in ((40, 12801), (77, 13001), (2056, 12810)):
        x, w, b, r = case(rows, n_in, n_out, dtype, seed=n_in)
        check_forward(lbp, x, w, b, r, "relu", f"few rows {rows} {n_in} {n_out} {dtype}")
    print(f"few rows {rows} {dtype}", flush=True)


@pytest.mark.parametrize("size, dtype", [((4090, 4088, 4080), BF16), ((4090, 4088, 4080), F16), ((4091, 1001, 4085), BF16),
                                         ((8190, 72, 2056), F16), ((4090, 400, 4088), F32), ((2041, 1019, 2045), F32),
                                         ((70, 8192, 72), BF16), ((90, 4100, 260), F32), ((2050, 2000, 1030), BF16)],
                         ids=str)
def test_large_products(lbp, size, dtype):
    """Sizes that take the largest tiles (all three products) and split reductions, none of them a
    whole number of tiles or stages."""
    rows, n_in, n_out = size
    print(f"large {size} {dtype}", flush=True)
    x, w, b, r = case(*size, dtype, seed=70)
    check_forward(lbp, x, w, b, r, "relu", f"large {size}")
    dy = normal(gen(71), rows, n_out, std=rows ** -0.5, dtype=dtype)
    check_backward(lbp, dy, x, w, None, "none", f"large {size}")
    check_backward(lbp, dy, x, w, r, "silu", f"large {size}")


@pytest.mark.parametrize("size, dtype", [((1030, 2050, 2000), F16), ((1021, 2047, 2045), F32), ((300, 701, 5000), BF16),
                                         ((2047, 1000, 1033), F32)], ids=str)
def test_gradients_alone_and_together(lbp, size, dtype):
    """Both products by one launch, with wide and narrow tiles, and the column sums beside them."""
    rows, n_in, n_out = size
    print(f"together {size} {dtype}", flush=True)
    x, w, b, r = case(*size, dtype, seed=80)
    dy = normal(gen(81), rows, n_out, std=rows ** -0.5, dtype=dtype)
    out = check_backward(lbp, dy, x, w, r, "gelu", f"together {size}")
    for k, name in enumerate(("want_x", "want_weight", "want_bias")):
        flags = dict(want_x=False, want_weight=False, want_bias=False)
        flags[name] = True
        one = lbp.linear_backward(dy, x, w, act="gelu", saved=r, **flags)
        assert torch.equal(one[k], out[k]), name


def test_refusals_of_the_binding(lbp):
    x, w, b, r = case(6, 8, 5, F32)
    for call, text in (
            (lambda: lbp.linear(x, w.t()), "weight"), (lambda: lbp.linear(x.t(), w), "contiguous|weight"),
            (lambda: lbp.linear(x, w.half()), "weight"), (lambda: lbp.linear(x, w.cpu()), "weight"),
            (lambda: lbp.linear(x, w, b[:4]), "bias"), (lambda: lbp.linear(x, w, b, r[:5]), "residual"),
            (lambda: lbp.linear(x, w, act="tanh"), "act"), (lambda: lbp.linear(x[0], w), "matrices"),
            (lambda: lbp.linear(x, w, out=r[:, :4]), "out"), (lambda: lbp.linear(x.double(), w.double()), "float32"),
            (lambda: lbp.linear_backward(r, x, w, act="relu"), "saved"),
            (lambda: lbp.linear_backward(r, x, w, saved=r), "saved"),
            (lambda: lbp.linear_backward(r[:5], x, w), "dy"),
            (lambda: lbp.linear_backward(r, x, w, act="gelu", saved=r.half()), "saved")):
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(lbp.VBError, match="nothing to compute"):
        lbp.linear_backward(r, x, w, want_x=False, want_weight=False, want_bias=False)
    with pytest.raises(lbp.VBError, match="leading dimension"):        # a broadcast residual has no rows
        lbp.linear(x, w, b, r[:1].expand(6, 5))
