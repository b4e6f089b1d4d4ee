"""The training operators in float64 (plain torch, any device), and the error
bounds their float32 / 16-bit evaluation has to keep.

Bounds are first-order worst cases for any order of summation: a float32 sum of
n products is within n 2^-24 of sum |a||b|, and rounding to a type adds half a
unit in its last place.
"""
import math

import torch

U32 = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # 2^-(significand bits)
# half the spacing of the subnormal numbers (float32's also covers a flush to zero)
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}
# error of an activation's factor: expf / erfcf to a few units for float32 data,
# the hardware exponential (2^-20) for 16-bit data
ACT = {torch.float32: 2.0 ** -20, torch.bfloat16: 2.0 ** -18, torch.float16: 2.0 ** -18}


def act(v, name):
    if name == "relu":
        return torch.where(v > 0, v, torch.where(torch.isnan(v), v, torch.zeros_like(v)))
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "silu":
        return v * torch.sigmoid(v)
    return v


def act_grad(saved, name):
    if name == "relu":
        return (saved > 0).double()
    if name == "gelu":
        return torch.special.ndtr(saved) + saved * torch.exp(-saved * saved / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        q = torch.sigmoid(saved)
        return q + saved * q * (1 - q)
    return torch.ones_like(saved)


def mm(a, b):
    """Float64 product, with contiguous operands."""
    return torch.mm(a.double().contiguous(), b.double().contiguous())


def linear(x, w, bias, res, name):
    """(y, pre, their error bounds) in float64."""
    dt = x.dtype
    pre = mm(x, w.t())
    mag = mm(x.abs(), w.abs().t())
    for t in (bias, res):
        if t is not None:
            pre = pre + t.double()
            mag = mag + t.double().abs()
    y = act(pre, name)
    e = (x.shape[1] + 4) * U32 * mag
    ea = 1.13 * e + (ACT[dt] * pre.abs() if name in ("gelu", "silu") else 0.0)
    return y, pre, ea + UNIT[dt] * (y.abs() + ea) + TINY[dt], e + UNIT[dt] * (pre.abs() + e) + TINY[dt]


def linear_backward(dy, x, w, saved, name):
    """{name: (value, error bound)} in float64."""
    dt = x.dtype
    if name == "none":
        g = dy.double()
    elif name == "relu":
        g = torch.where(saved > 0, dy.double(), torch.zeros_like(dy, dtype=torch.float64))
    else:
        g = dy.double() * act_grad(saved.double(), name)
    smooth = name in ("gelu", "silu")
    # g itself, and g as an operand of the products
    eg = (ACT[dt] * dy.double().abs() * (1 + (saved.double().abs() if smooth else 0))) if smooth else torch.zeros_like(g)
    eo = eg + ((UNIT[dt] if dt != torch.float32 else U32) * g.abs() + TINY[dt] if smooth else 0.0)

    def product(a, ea, b, k):
        v = mm(a, b)
        e = mm(ea, b.abs()) + (k + 4) * U32 * mm(a.abs(), b.abs())
        return v, e + UNIT[dt] * (v.abs() + e) + TINY[dt]

    rows, n_out = g.shape
    db = g.sum(0)
    edb = eg.sum(0) + (rows + 4) * U32 * g.abs().sum(0)
    return {"dx": product(g, eo, w, n_out), "dweight": product(g.t(), eo.t(), x, rows),
            "dbias": (db, edb + UNIT[dt] * (db.abs() + edb) + TINY[dt]),
            "dresidual": (g, eg + UNIT[dt] * (g.abs() + eg) + TINY[dt])}


def cross_entropy(z, labels, ignore, eps, scale):
    """(loss, row_loss, dlogits) in float64, row by row from the definition."""
    rows, classes = z.shape
    row = torch.zeros(rows, dtype=torch.float64)
    grad = torch.zeros(rows, classes, dtype=torch.float64)
    labels = labels.cpu()
    zz = z.detach().double().cpu()
    use = [r for r in range(rows) if int(labels[r]) != ignore]
    n = max(len(use), 1)
    for r in use:
        t = int(labels[r])
        logp = torch.log_softmax(zz[r], 0)
        if not 0 <= t < classes:
            row[r] = math.nan
            grad[r] = math.nan
            continue
        row[r] = -(1 - eps) * logp[t] if eps < 1 else 0.0
        if eps > 0:
            row[r] = row[r] - eps * logp.mean()
        d = logp.exp() - eps / classes
        d[t] -= 1 - eps
        grad[r] = d * (scale / n)
    return (row.sum() / n) if use else torch.tensor(0.0, dtype=torch.float64), row, grad


def assert_within(got, want, bound, what):
    """got within bound of want; infinities and NaN exactly where want has them."""
    g = got.double()
    w = want.to(g.device)
    b = bound.to(g.device) if torch.is_tensor(bound) else torch.full_like(w, bound)
    assert g.shape == w.shape, (what, g.shape, w.shape)
    finite = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w)), f"{what}: NaN in other places"
    inf = torch.isinf(w)
    assert torch.equal(g[inf], w[inf]), f"{what}: infinities differ"
    over = ((g - w).abs() > b) & finite
    if over.any():
        ratio = ((g - w).abs() / b)
        ratio[~finite] = 0
        i = int(ratio.argmax())
        raise AssertionError(f"{what}: {int(over.sum())}/{over.numel()} outside the bound; worst at {i}: "
                             f"{g.flatten()[i].item()!r} for {w.flatten()[i].item()!r}, bound {b.flatten()[i].item():.3g}")
