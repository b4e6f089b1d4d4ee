"""The 16-bit backward pass with GELU and SiLU holds the gradient of the pre-activation in
more bits than its operands' type has (unless asked not to): against float64, at tolerances
that a single rounding of it does not keep."""
import itertools

import pytest
import torch

import train_reference as ref
from helpers import ensure_built

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
# relative error of the two numbers that stand for g, and its floor (float16: half the spacing
# of the subnormal numbers, 2^-25, times the low part's 2^(1 - 11))
SPLIT = {BF16: 2.0 ** -16, F16: 2.0 ** -22}
FLOOR = {BF16: 2.0 ** -126, F16: 2.0 ** -35}


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def normal(seed, *shape, std=1.0, dtype=F16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def case(rows, n_in, n_out, dtype, seed=0):
    return (normal(seed, rows, n_out, dtype=dtype), normal(seed + 1, rows, n_in, dtype=dtype),
            normal(seed + 2, n_out, n_in, std=n_in ** -0.5, dtype=dtype), normal(seed + 3, rows, n_out, dtype=dtype))


def want(dy, x, w, saved, act):
    """{name: (value, bound)}: g = dy act' within the activation's error and the split's, float32
    sums over both parts, one rounding of the result."""
    dt = x.dtype
    g = dy.double() * ref.act_grad(saved.double(), act)
    eg = ref.ACT[dt] * dy.double().abs() * (1 + saved.double().abs()) + SPLIT[dt] * g.abs() + FLOOR[dt]

    def product(a, ea, b):
        v = ref.mm(a, b)
        e = ref.mm(ea, b.abs()) + (2 * a.shape[1] + 8) * ref.U32 * ref.mm(a.abs(), b.abs())
        return v, e + ref.UNIT[dt] * (v.abs() + e) + ref.TINY[dt]

    return {"dx": product(g, eg, w), "dweight": product(g.t(), eg.t(), x)}


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("size", [(1, 64, 64), (16, 100, 10), (17, 33, 65), (65, 100, 129), (300, 1000, 130), (70, 4096, 72),
                                  (1037, 333, 257), (2050, 2000, 1030), (4090, 2040, 2056)], ids=str)
def test_products_of_the_unrounded_gradient(lbp, size, dtype, act):
    print(f"backward bits {size} {dtype} {act}", flush=True)
    dy, x, w, saved = case(*size, dtype)
    bounds = want(dy, x, w, saved, act)
    dx, dw, db, dr = lbp.linear_backward(dy, x, w, act=act, saved=saved, want_residual=True)
    ref.assert_within(dx, *bounds["dx"], f"{size} dx")
    ref.assert_within(dw, *bounds["dweight"], f"{size} dweight")
    # the same bits alone, and every gradient the same again
    assert torch.equal(lbp.linear_backward(dy, x, w, act=act, saved=saved, want_weight=False, want_bias=False)[0], dx)
    assert torch.equal(lbp.linear_backward(dy, x, w, act=act, saved=saved, want_x=False, want_bias=False)[1], dw)
    # rounded where the caller asks for it: dbias and dresidual do not change
    rounded = lbp.linear_backward(dy, x, w, act=act, saved=saved, want_residual=True, round_g=True)
    assert torch.equal(rounded[2], db) and torch.equal(rounded[3], dr)
    old = ref.linear_backward(dy, x, w, saved, act)
    for k, name in enumerate(("dx", "dweight")):
        ref.assert_within(rounded[k], *old[name], f"{size} {name} of the rounded gradient")


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_unaligned_operands(lbp, dtype):
    rows, n_in, n_out = 203, 251, 137
    dy, x, w, saved = case(rows, n_in, n_out, dtype, seed=9)

    def odd(t):
        buf = torch.full((t.shape[0], t.shape[1] + 4), float("nan"), dtype=dtype, device="cuda")
        buf[:, 1:1 + t.shape[1]] = t
        return buf[:, 1:1 + t.shape[1]]

    dx, dw, _, _ = lbp.linear_backward(odd(dy), odd(x), odd(w), act="gelu", saved=odd(saved))
    bounds = want(dy, x, w, saved, "gelu")
    ref.assert_within(dx, *bounds["dx"], "unaligned dx")
    ref.assert_within(dw, *bounds["dweight"], "unaligned dweight")


def test_float16_gradients_at_both_ends_of_the_range(lbp):
    """g beyond float16's largest number (act' is above 1 there), and below its smallest."""
    rows, n_in, n_out = 64, 40, 48
    w = torch.full((n_out, n_in), 2.0 ** -9, dtype=F16, device="cuda")
    for act, at in (("gelu", 1.5), ("silu", 2.5)):
        saved = torch.full((rows, n_out), at, dtype=F16, device="cuda")
        dy = torch.full((rows, n_out), 65504.0, dtype=F16, device="cuda")
        x = torch.full((rows, n_in), 2.0 ** -9, dtype=F16, device="cuda")
        bounds = want(dy, x, w, saved, act)
        dx, dw, _, _ = lbp.linear_backward(dy, x, w, act=act, saved=saved)
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
        ref.assert_within(dx, *bounds["dx"], f"large {act} dx")
        ref.assert_within(dw, *bounds["dweight"], f"large {act} dweight")
    dy = torch.full((rows, n_out), 3 * 2.0 ** -24, dtype=F16, device="cuda")
    saved = torch.full((rows, n_out), -0.5, dtype=F16, device="cuda")
    x = torch.full((rows, n_in), 1024.0, dtype=F16, device="cuda")
    bounds = want(dy, x, w, saved, "gelu")
    dw = lbp.linear_backward(dy, x, w, act="gelu", saved=saved)[1]
    ref.assert_within(dw, *bounds["dweight"], "small dweight")


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_infinities_and_nan(lbp, dtype):
    """An infinity or NaN of one operand reaches what the formula says, with its sign."""
    rows, n_in, n_out = 150, 130, 140
    dy, x, w, saved = case(rows, n_in, n_out, dtype, seed=20)
    sign = torch.where(dy < 0, -1.0, 1.0).to(dtype)
    dy = sign * dy.abs().clamp_min(0.125)
    saved = saved.abs() + 0.5           # g of dy's sign and well away from zero
    for which, value in itertools.product(("x", "weight", "dy"), (float("inf"), float("-inf"), float("nan"))):
        d, a, b = dy.clone(), x.clone(), w.clone()
        {"x": a, "weight": b, "dy": d}[which][7, 3] = value
        dx, dw, db, _ = lbp.linear_backward(d, a, b, act="gelu", saved=saved)
        bounds = want(d, a, b, saved, "gelu")
        ref.assert_within(dx, *[t.nan_to_num(0, 0, 0) if i else t for i, t in enumerate(bounds["dx"])], f"{which} {value} dx")
        ref.assert_within(dw, *[t.nan_to_num(0, 0, 0) if i else t for i, t in enumerate(bounds["dweight"])],
                          f"{which} {value} dweight")


def test_kept_workspace_serves_every_activation(lbp):
    for size in ((5, 70, 40), (90, 2050, 260), (700, 800, 900)):
        for dtype in (torch.float32, BF16, F16):
            dy, x, w, saved = case(*size, dtype, seed=30)
            ws = lbp.linear_workspace(x, w, backward=True)
            for act in ("none", "relu", "gelu", "silu"):
                s = None if act == "none" else saved
                for round_g in (False, True):
                    a = lbp.linear_backward(dy, x, w, act=act, saved=s, want_residual=True, round_g=round_g)
                    b = lbp.linear_backward(dy, x, w, act=act, saved=s, want_residual=True, round_g=round_g, ws=ws)
                    assert all(torch.equal(p, q) for p, q in zip(a, b)), (size, dtype, act, round_g)
                    if act in ("none", "relu") or dtype == torch.float32:
                        c = lbp.linear_backward(dy, x, w, act=act, saved=s, want_residual=True, round_g=not round_g)
                        assert all(torch.equal(p, q) for p, q in zip(a, c)), (size, dtype, act)
