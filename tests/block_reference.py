"""Layer norm, the gated linear layer and dropout in float64 (plain torch, any device), and
the error bounds that their float32 / 16-bit evaluation has to keep: first-order worst cases
for any order of summation, as in train_reference."""
import numpy as np
import torch

from train_reference import ACT, TINY, U32, UNIT, act, act_grad, mm

# what g loses as an operand of the products: nothing in float32, else the two parts' 2^-2p
SPLIT = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22}


def rounded(v, e, dt):
    """Bound of a value v, computed within e and rounded to dt."""
    return e + UNIT[dt] * (v.abs() + e) + TINY[dt]


def layer_norm(x, w, b, eps):
    """{name: (value, bound)} of y, mean, rstd."""
    dt, n = x.dtype, x.shape[1]
    x = x.double()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = (c * c).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    wd = torch.ones_like(c[:1]) if w is None else w.double()
    y = c * rstd * wd
    # a first mean from differences s to the first element, off by (n + 4) u mean s and its own
    # rounding; differences d from that (u d), and the mean of those
    s = (x - x[:, :1]).abs().mean(1, keepdim=True)
    first = (n + 4) * U32 * s + 2 * U32 * mean.abs()
    d = c.abs() + first
    em = (n + 4) * U32 * d.mean(1, keepdim=True)
    ec = 2 * U32 * d + em
    ev = (n + 8) * U32 * (d * d).mean(1, keepdim=True)
    er = 0.5 * ev / (var + eps) + 4 * U32                       # relative, of rstd
    ey = (ec * rstd + c.abs() * rstd * (er + 3 * U32)) * wd.abs()
    if b is not None:
        y = y + b.double()
    ey = ey + 2 * U32 * (y.abs() + (c * rstd * wd).abs())
    return {"y": (y, rounded(y, ey, dt)), "mean": (mean[:, 0], (em + 2 * U32 * (mean.abs() + first))[:, 0] + TINY[torch.float32]),
            "rstd": (rstd[:, 0], (rstd * (er + U32))[:, 0])}


def layer_norm_backward(dy, x, mean, rstd, w, res):
    """{name: (value, bound)} of dx, dweight, dbias, from the given statistics."""
    dt, (rows, n) = x.dtype, x.shape
    dy, r = dy.double(), rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    wd = torch.ones_like(xh[:1]) if w is None else w.double()
    g = dy * wd
    level, along = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - level - xh * along)
    e_level = (n + 4) * U32 * g.abs().mean(1, keepdim=True)
    e_along = (n + 8) * U32 * (g * xh).abs().mean(1, keepdim=True)
    e = r * (e_level + xh.abs() * e_along + 6 * U32 * (g.abs() + level.abs() + 2 * (xh * along).abs()))
    if res is not None:
        dx = dx + res.double()
        e = e + 2 * U32 * (dx.abs() + res.double().abs())
    dw, db = (dy * xh).sum(0), dy.sum(0)
    edw = (rows + 8) * U32 * (dy * xh).abs().sum(0)
    edb = (rows + 4) * U32 * dy.abs().sum(0)
    return {"dx": (dx, rounded(dx, e, dt)), "dweight": (dw, rounded(dw, edw, dt)), "dbias": (db, rounded(db, edb, dt))}


def gated(x, w, b, name):
    """{name: (value, bound)} of y and pre."""
    dt, n = x.dtype, w.shape[0] // 2
    pre, mag = mm(x, w.t()), mm(x.abs(), w.abs().t())
    if b is not None:
        pre, mag = pre + b.double(), mag + b.double().abs()
    e = (x.shape[1] + 4) * U32 * mag
    gate, up, eg, eu = pre[:, :n], pre[:, n:], e[:, :n], e[:, n:]
    a = act(gate, name)
    ea = 1.13 * eg + (ACT[dt] * gate.abs() if name in ("gelu", "silu") else 0.0)
    y = a * up
    ey = ea * up.abs() + a.abs() * eu + ea * eu + 2 * U32 * y.abs()
    return {"y": (y, rounded(y, ey, dt)), "pre": (pre, rounded(pre, e, dt))}


def gated_backward(dy, x, w, pre, name, round_g=False):
    """{name: (value, bound)} of dx, dweight, dbias."""
    dt, n = x.dtype, w.shape[0] // 2
    dy, gate, up = dy.double(), pre[:, :n].double(), pre[:, n:].double()
    smooth = ACT[dt] if name in ("gelu", "silu") else 0.0
    slope = (gate > 0).double() if name == "relu" else act_grad(gate, name)
    g = torch.cat([torch.where(slope == 0, torch.zeros_like(dy), dy * up * slope) if name == "relu" else dy * up * slope,
                   dy * act(gate, name)], 1)
    eg = torch.cat([smooth * (1 + gate.abs()) * (dy * up).abs(), smooth * (dy * gate).abs()], 1) + 3 * U32 * g.abs()
    eo = eg + (UNIT[dt] if round_g else SPLIT[dt]) * g.abs() + TINY[dt]

    def product(a, ea, b, k):
        v = mm(a, b)
        e = mm(ea, b.abs()) + (2 * k + 8) * U32 * mm(a.abs(), b.abs())
        return v, rounded(v, e, dt)

    rows = x.shape[0]
    db = g.sum(0)
    return {"dx": product(g, eo, w, 2 * n), "dweight": product(g.t(), eo.t(), x, rows),
            "dbias": (db, rounded(db, eg.sum(0) + (rows + 4) * U32 * g.abs().sum(0), dt))}


def philox(counter, key, rounds=7):
    """Four words of Philox4x32 for one counter and key, in Python's integers: (c0, c1, c2, c3), (k0, k1)."""
    c, k, m = list(counter), list(key), 0xFFFFFFFF
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def kept(rows, n, p, seed, offset, first_row=0):
    """The mask of `rows` rows from first_row on, as a CPU tensor (numpy's unsigned integers)."""
    u = np.uint64
    m, h = u(0xFFFFFFFF), u(32)
    quads = (n + 3) // 4
    at = np.arange(first_row * quads, (first_row + rows) * quads, dtype=u)
    c = [at & m, at >> h, np.full_like(at, offset & 0xFFFFFFFF), np.full_like(at, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(7):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> h) ^ c[1] ^ u(k[0]), b & m, (a >> h) ^ c[3] ^ u(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(c, 1).reshape(rows, 4 * quads)[:, :n]
    return torch.from_numpy(words >= u(round(p * 2 ** 32)))


def dropout(x, p, mask, res):
    """(value, bound)."""
    dt = x.dtype
    drop = round(p * 2 ** 32)
    scale = 2 ** 32 / (2 ** 32 - drop) if drop < 2 ** 32 else 0.0
    y = torch.where(mask.to(x.device), x.double() * scale, torch.zeros((), dtype=torch.float64, device=x.device))
    e = 2 * U32 * y.abs()
    if res is not None:
        y = y + res.double()
    return y, rounded(y, e + U32 * y.abs(), dt)
