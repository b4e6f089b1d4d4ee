"""Cases of the operators around a feed-forward block's linear layers: layer norm and its
backward pass, the gated linear layer (two projections, the activation of one times the
other) and its backward pass, and dropout from counted random numbers.

With `own` false, `run` computes the plain forms in elementary torch operations (float32,
rounded once at the end); with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


def _lbp():
    import linear_bound_propagation_amd as lbp
    return lbp


# --------------------------------------------------------------------------
# cases

def listed():
    return [
        # Normalising a hidden layer of the 784-100-100-10 network, 16 inputs: latency counts.
        dict(name="norm_mlp_f32", op="norm", rows=16, n=100, dtype="f32"),
        # A long prompt (or a training batch) before a feed-forward block.
        dict(name="norm_large_bf16", op="norm", rows=8192, n=8192, dtype="bf16"),
        # Training the norm of a pre-norm block, 8192 tokens: the skip connection's gradient comes in.
        dict(name="norm_backward_bf16", op="norm_backward", rows=8192, n=4096, dtype="bf16", residual=True),
        # A last, incomplete batch, sizes that divide by nothing.
        dict(name="norm_backward_ragged_f16", op="norm_backward", rows=1037, n=2001, dtype="f16", residual=False),
        # One token through the gate and the widening projection: the weights are read once.
        dict(name="gated_token_bf16", op="gated", rows=1, n_in=4096, n_out=16384, dtype="bf16", act="silu", keep=False),
        # A few tokens of a serving batch, sizes that divide by nothing.
        dict(name="gated_few_ragged_f16", op="gated", rows=7, n_in=5001, n_out=3999, dtype="f16", act="gelu",
             keep=False),
        # Training on 4096 tokens, forward: large matrix products; both projections are kept.
        dict(name="gated_large_bf16", op="gated", rows=4096, n_in=4096, n_out=8192, dtype="bf16", act="silu",
             keep=True),
        # The same, backward.
        dict(name="gated_backward_bf16", op="gated_backward", rows=4096, n_in=4096, n_out=8192, dtype="bf16",
             act="silu"),
        # Training a gated layer of a 1024-wide float32 network.
        dict(name="gated_backward_f32", op="gated_backward", rows=2048, n_in=1024, n_out=1024, dtype="f32", act="gelu"),
        # Dropout of a hidden layer of the 784-100-100-10 network: latency counts.
        dict(name="dropout_mlp_f32", op="dropout", rows=128, n=100, dtype="f32", p=0.5, residual=False),
        # What a feed-forward block of 8192 tokens gives, dropped in part and added to the residual stream.
        dict(name="dropout_large_bf16", op="dropout", rows=8192, n=8192, dtype="bf16", p=0.1, residual=True),
        # Its backward pass: the gradient through the same mask.
        dict(name="dropout_backward_bf16", op="dropout", rows=8192, n=4096, dtype="bf16", p=0.1, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _sizes(rng, budget, *ranges):
    while True:
        sizes = [_log(rng, lo, hi) for lo, hi in ranges]
        if math.prod(sizes) <= budget:
            return sizes


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "gated", "gated", "gated_backward", "gated_backward", "dropout"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op.startswith("gated"):
        # a single token to a long prompt; float32 layers as small as the MLP's
        budget = 2 ** 34 if dtype == "f32" else 2 ** 36
        rows, n_in, n_out = _sizes(rng, budget, (1, 8192), (10, 8192), (10, 16384))
        case = dict(op=op, rows=rows, n_in=n_in, n_out=n_out, dtype=dtype,
                    act=rng.choice(["none", "relu", "gelu", "silu", "silu"]))
        if op == "gated":
            case["keep"] = rng.random() < 0.5
        return case
    # one row to a long prompt, the narrowest layer to a wide one
    rows, n = _sizes(rng, 2 ** 26 if dtype != "f32" else 2 ** 25, (1, 16384), (10, 16384))
    case = dict(op=op, rows=rows, n=n, dtype=dtype)
    if op == "norm_backward":
        case["residual"] = rng.random() < 0.5
    if op == "dropout":
        case["p"] = rng.choice([0.1, 0.1, 0.5, 0.02])
        case["residual"] = rng.random() < 0.5
    return case


# --------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    state = dict(case)
    rows = case["rows"]
    # gradients of a mean over the rows; float16 ones carry a loss scale
    grad_std = 1.0 if case["dtype"] == "f16" else 1.0 / rows
    if case["op"].startswith("norm"):
        n = case["n"]
        # a residual stream: off zero, and of another size from channel to channel
        channels = 0.5 + 2 * torch.rand(n, generator=gen, device="cuda")
        state["x"] = ((torch.randn(rows, n, generator=gen, device="cuda") + 0.3) * channels).to(dtype)
        state["weight"] = normal(n, std=0.1, mean=1.0)
        if case["op"] == "norm":
            state["bias"] = normal(n, std=0.1)
            return state
        state["dy"] = normal(rows, n, std=grad_std)
        state["dres"] = normal(rows, n, std=grad_std) if case["residual"] else None
        # what the forward pass kept
        mean, var = [], []
        for part in state["x"].split(1024):
            part = part.double()
            mean.append(part.mean(1))
            var.append(((part - mean[-1][:, None]) ** 2).mean(1))
        state["mean"] = torch.cat(mean).float()
        state["rstd"] = (torch.cat(var) + EPS).rsqrt().float()
        if own:
            state["ws"] = _lbp().layer_norm_workspace(state["x"])
    elif case["op"].startswith("gated"):
        n_in, n_out = case["n_in"], case["n_out"]
        # weights N(0, 1/fan_in): the gate's rows, then the other projection's
        state["weight"] = normal(2 * n_out, n_in, std=n_in ** -0.5)
        state["x"] = normal(rows, n_in)
        if case["op"] == "gated":
            state["bias"] = normal(2 * n_out, std=0.1)
        else:
            state["pre"] = normal(rows, 2 * n_out)
            state["dy"] = normal(rows, n_out, std=grad_std)
        if own:
            state["ws"] = _lbp().gated_linear_workspace(state["x"], state["weight"],
                                                        backward=case["op"] == "gated_backward")
    else:
        state["x"] = normal(rows, case["n"])
        state["res"] = normal(rows, case["n"]) if case["residual"] else None
        # the step of a long training is the offset; it counts past 32 bits
        state["seed"] = seed * 0x9E3779B97F4A7C15 % 2 ** 64
        state["offset"] = 2 ** 33 + 7 * seed
    return state


# --------------------------------------------------------------------------
# one pass

def _act(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _act_grad(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "gelu":
        phi = torch.exp(-0.5 * v * v) * (2 * math.pi) ** -0.5
        return 0.5 * (1 + torch.erf(v * 0.5 ** 0.5)) + v * phi
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    return torch.ones_like(v)


def _random_words(rows, n, seed, offset, device):
    """[rows][n] random 32-bit words (int64): word c % 4 of Philox4x32-7 (Salmon et al., 2011) with
    key `seed` and counter (row * ceil(n / 4) + c // 4, offset), 64 bits each."""
    low = 0xFFFFFFFF
    quads = (n + 3) // 4
    at = torch.arange(rows * quads, dtype=torch.int64, device=device)
    c = [at & low, at >> 32, torch.full_like(at, offset & low), torch.full_like(at, offset >> 32)]
    k = [seed & low, seed >> 32]
    for _ in range(7):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57     # the 64 bits of a product, whatever their sign
        c = [(b >> 32 & low) ^ c[1] ^ k[0], b & low, (a >> 32 & low) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return torch.stack(c, 1).reshape(rows, 4 * quads)[:, :n]


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    dt = state["x"].dtype
    if op == "norm":
        x = state["x"].float()
        mean = x.mean(1)
        x = x - mean[:, None]
        rstd = 1 / torch.sqrt((x * x).mean(1) + EPS)
        y = x * rstd[:, None] * state["weight"].float() + state["bias"].float()
        return {"y": y.to(dt), "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        dy, rstd = state["dy"].float(), state["rstd"][:, None]
        xh = (state["x"].float() - state["mean"][:, None]) * rstd
        g = dy * state["weight"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if state["dres"] is not None:
            dx = dx + state["dres"].float()
        return {"dx": dx.to(dt), "dweight": (dy * xh).sum(0).to(dt), "dbias": dy.sum(0).to(dt)}
    if op == "gated":
        n = state["n_out"]
        pre = state["x"].float() @ state["weight"].float().t() + state["bias"].float()
        out = {"y": (_act(pre[:, :n], state["act"]) * pre[:, n:]).to(dt)}
        if state["keep"]:
            out["pre"] = pre.to(dt)
        return out
    if op == "gated_backward":
        n = state["n_out"]
        gate, up, dy = state["pre"][:, :n].float(), state["pre"][:, n:].float(), state["dy"].float()
        g = torch.cat([dy * up * _act_grad(gate, state["act"]), dy * _act(gate, state["act"])], 1)
        return {"dx": (g @ state["weight"].float()).to(dt), "dweight": (g.t() @ state["x"].float()).to(dt),
                "dbias": g.sum(0).to(dt)}
    rows, n = state["x"].shape
    keep = _random_words(rows, n, state["seed"], state["offset"], state["x"].device) >= round(state["p"] * 2 ** 32)
    y = torch.where(keep, state["x"].float() * (1 / (1 - state["p"])), torch.zeros((), device=state["x"].device))
    if state["res"] is not None:
        y = y + state["res"].float()
    return {"y": y.to(dt)}


def _run_own(state):
    lbp = _lbp()
    op = state["op"]
    if op == "norm":
        y, mean, rstd = lbp.layer_norm(state["x"], state["weight"], state["bias"], eps=EPS, want_stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        dx, dw, db = lbp.layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"],
                                             dresidual=state["dres"], ws=state["ws"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "gated":
        y = lbp.gated_linear(state["x"], state["weight"], state["bias"], act=state["act"], want_pre=state["keep"],
                             ws=state["ws"])
        return {"y": y[0], "pre": y[1]} if state["keep"] else {"y": y}
    if op == "gated_backward":
        dx, dw, db = lbp.gated_linear_backward(state["dy"], state["x"], state["weight"], state["pre"],
                                               act=state["act"], ws=state["ws"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    return {"y": lbp.dropout(state["x"], state["p"], state["seed"], state["offset"], residual=state["res"])}


# --------------------------------------------------------------------------
# the least work of a pass, and its value in 64 bits

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    m = case["rows"]
    if case["op"] == "norm":
        n = case["n"]
        return {"bytes": size * (2 * m * n + 2 * n) + 8 * m, "flops": 8 * m * n}
    if case["op"] == "norm_backward":
        n = case["n"]
        return {"bytes": size * (m * n * (3 + case["residual"]) + 3 * n) + 8 * m, "flops": 13 * m * n}
    if case["op"] == "gated":
        k, n = case["n_in"], case["n_out"]
        return {"bytes": size * (m * k + 2 * n * k + 2 * n + m * n * (1 + 2 * case["keep"])), "flops": 4 * m * n * k}
    if case["op"] == "gated_backward":
        k, n = case["n_in"], case["n_out"]
        return {"bytes": size * (2 * m * k + 4 * n * k + 2 * n + 3 * m * n), "flops": 8 * m * n * k}
    return {"bytes": size * m * case["n"] * (2 + case["residual"]), "flops": (1 + case["residual"]) * m * case["n"]}


def _kept(rows, n, seed, offset, p):
    """Which elements stay, on the host in unsigned 64-bit arithmetic."""
    u, low, half = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    quads = (n + 3) // 4
    keep = np.empty((rows, 4 * quads), dtype=bool)
    step = max(1, (1 << 21) // quads)
    for r0 in range(0, rows, step):
        r1 = min(rows, r0 + step)
        at = np.arange(r0 * quads, r1 * quads, dtype=u)
        x, y = at & low, at >> half
        z, w = np.full_like(at, offset % 2 ** 32), np.full_like(at, offset // 2 ** 32)
        for i in range(7):
            ka = u((seed % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32)
            kb = u((seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32)
            s, t = x * u(0xD2511F53), z * u(0xCD9E8D57)
            x, y, z, w = (t >> half) ^ y ^ ka, t & low, (s >> half) ^ w ^ kb, s & low
        words = keep[r0:r1].reshape(-1, 4)
        for j, word in enumerate((x, y, z, w)):
            words[:, j] = word >= u(round(p * 2 ** 32))
    return keep[:, :n]


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, 1, correction=0)
        y = (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
        return {"y": torch.addcmul(s["bias"].double(), y, s["weight"].double()), "mean": mean,
                "rstd": (var + EPS) ** -0.5}
    if case["op"] == "norm_backward":
        m, r, n = s["mean"].double()[:, None], s["rstd"].double()[:, None], case["n"]
        dy = s["dy"].double()
        dbias = dy.sum(0)
        norm = x.sub_(m).mul_(r)
        dweight = torch.mul(dy, norm).sum(0)
        dy *= s["weight"].double()
        along, level = (dy * norm).sum(1, keepdim=True) / n, dy.sum(1, keepdim=True) / n
        dx = dy.sub_(norm.mul_(along)).sub_(level).mul_(r)
        if s["dres"] is not None:
            dx += s["dres"].double()
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if case["op"] == "gated":
        gate, up = (torch.mm(x, w.double().t().contiguous()) + b.double()
                    for w, b in zip(s["weight"].chunk(2), s["bias"].chunk(2)))
        y = up * {"none": lambda: gate, "relu": lambda: torch.clamp_min(gate, 0), "silu": lambda: gate * torch.sigmoid(gate),
                  "gelu": lambda: gate * torch.special.ndtr(gate)}[case["act"]]()
        return {"y": y, "pre": torch.cat([gate, up], 1)} if case["keep"] else {"y": y}
    if case["op"] == "gated_backward":
        gate, up = (t.double() for t in s["pre"].chunk(2, 1))
        dy = s["dy"].double()
        if case["act"] == "none":
            value, slope = gate, torch.ones_like(gate)
        elif case["act"] == "relu":
            value, slope = torch.clamp_min(gate, 0), (gate > 0).double()
        elif case["act"] == "gelu":
            cdf = torch.special.ndtr(gate)
            value, slope = gate * cdf, cdf + gate * torch.exp(-gate * gate / 2) / math.sqrt(2 * math.pi)
        else:
            q = torch.sigmoid(gate)
            value, slope = gate * q, q + gate * q * torch.sigmoid(-gate)
        parts = (dy * up * slope, dy * value)
        dx = sum(torch.mm(g, w.double()) for g, w in zip(parts, s["weight"].chunk(2)))
        return {"dx": dx, "dweight": torch.cat([torch.mm(g.t().contiguous(), x) for g in parts]),
                "dbias": torch.cat([g.sum(0) for g in parts])}
    keep = torch.from_numpy(_kept(*x.shape, s["seed"], s["offset"], case["p"])).to(x.device)
    y = torch.zeros_like(x)
    y[keep] = x[keep] / (1 - case["p"])
    return {"y": y if s["res"] is None else y + s["res"].double()}
