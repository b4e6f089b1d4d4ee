"""A pre-norm feed-forward block of the training operators, forward and backward as a user's
program runs it: x + dropout(linear(gated_linear(layer_norm(x))))."""
import pytest
import torch

import block_reference as ref
import train_reference as tref
from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def parameters(width, hidden, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*s, std=1.0, mean=0.0):
        return (torch.randn(*s, generator=g, device="cuda") * std + mean).to(dtype)

    return dict(norm_w=normal(width, std=0.1, mean=1.0), norm_b=normal(width, std=0.1),
                gated_w=normal(2 * hidden, width, std=width ** -0.5), gated_b=normal(2 * hidden, std=0.1),
                down_w=normal(width, hidden, std=hidden ** -0.5), down_b=normal(width, std=0.1))


class Block:
    def __init__(self, lbp, params, p, seed):
        self.lbp, self.p, self.drop, self.seed = lbp, params, p, seed

    def forward(self, x, offset):
        lbp, p = self.lbp, self.p
        h, mean, rstd = lbp.layer_norm(x, p["norm_w"], p["norm_b"], want_stats=True)
        a, pre = lbp.gated_linear(h, p["gated_w"], p["gated_b"], want_pre=True)
        o = lbp.linear(a, p["down_w"], p["down_b"])
        y = lbp.dropout(o, self.drop, self.seed, offset, residual=x, out=o)
        return y, (x, mean, rstd, h, pre, a, offset)

    def backward(self, dy, saved):
        lbp, p = self.lbp, self.p
        x, mean, rstd, h, pre, a, offset = saved
        do = lbp.dropout(dy, self.drop, self.seed, offset)
        da, down_w, down_b, _ = lbp.linear_backward(do, a, p["down_w"])
        dh, gated_w, gated_b = lbp.gated_linear_backward(da, h, p["gated_w"], pre)
        dx, norm_w, norm_b = lbp.layer_norm_backward(dh, x, mean, rstd, p["norm_w"], dresidual=dy, dx=dh)
        return dx, dict(norm_w=norm_w, norm_b=norm_b, gated_w=gated_w, gated_b=gated_b, down_w=down_w, down_b=down_b)


def formula(x, p, mask, drop):
    """The block in float64, for autograd."""
    c = x - x.mean(1, keepdim=True)
    h = c * ((c * c).mean(1, keepdim=True) + 1e-5) ** -0.5 * p["norm_w"] + p["norm_b"]
    gate, up = (h @ p["gated_w"].t() + p["gated_b"]).chunk(2, 1)
    o = (gate * torch.sigmoid(gate) * up) @ p["down_w"].t() + p["down_b"]
    return x + torch.where(mask, o / (1 - drop), torch.zeros_like(o))


@pytest.mark.parametrize("rows, width, hidden", [(1, 64, 100), (37, 100, 77), (300, 256, 513)])
def test_block_against_autograd(lbp, rows, width, hidden):
    """float32: each of the block's ten sums of K terms is off by at most (K + 8) 2^-24 of its terms'
    magnitudes, which exceed the values about tenfold here (random signs, K <= 1026): together
    10 * 1034 * 2^-24 * 10 = 2^-7.3 of the largest value at worst; 2^-9 is asked for."""
    params = parameters(width, hidden, torch.float32, 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x, dy = (torch.randn(rows, width, generator=g, device="cuda") for _ in range(2))
    block = Block(lbp, params, 0.2, 99)
    y, saved = block.forward(x, 2 ** 40)
    dx, grads = block.backward(dy, saved)
    mask = ref.kept(rows, width, 0.2, 99, 2 ** 40)
    leaves = {k: v.double().cpu().requires_grad_() for k, v in params.items()}
    xl = x.double().cpu().requires_grad_()
    out = formula(xl, leaves, mask, 0.2)
    out.backward(dy.double().cpu())

    def near(got, want, what):
        assert float((got.double().cpu() - want).abs().max()) <= 2.0 ** -9 * float(want.abs().max()), what

    near(y, out.detach(), "y")
    near(dx, xl.grad, "dx")
    for k in params:
        near(grads[k], leaves[k].grad, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_block_step_by_step(lbp, dtype):
    """16-bit types: every call of the block against float64 on the inputs that it got."""
    rows, width, hidden = 200, 264, 520
    params = parameters(width, hidden, dtype, 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x, dy = (torch.randn(rows, width, generator=g, device="cuda").to(dtype) for _ in range(2))
    p = params
    want = ref.layer_norm(x, p["norm_w"], p["norm_b"], float(torch.tensor(1e-5)))
    h, mean, rstd = lbp.layer_norm(x, p["norm_w"], p["norm_b"], want_stats=True)
    tref.assert_within(h, *want["y"], "norm")
    want = ref.gated(h, p["gated_w"], p["gated_b"], "silu")
    a, pre = lbp.gated_linear(h, p["gated_w"], p["gated_b"], want_pre=True)
    tref.assert_within(a, *want["y"], "gated")
    o = lbp.linear(a, p["down_w"], p["down_b"])
    mask = ref.kept(rows, width, 0.1, 5, 6)
    block = Block(lbp, params, 0.1, 5)
    y, saved = block.forward(x, 6)
    tref.assert_within(y, *ref.dropout(o, 0.1, mask, x), "dropout")
    assert torch.equal(saved[3], h) and torch.equal(saved[4], pre) and torch.equal(saved[5], a)
    dx, grads = block.backward(dy, saved)
    do = lbp.dropout(dy, 0.1, 5, 6)
    tref.assert_within(do, *ref.dropout(dy, 0.1, mask, None), "dropout backward")
    da, dw, db, _ = lbp.linear_backward(do, a, p["down_w"])
    back = ref.gated_backward(da, h, p["gated_w"], pre, "silu")
    dh = lbp.gated_linear_backward(da, h, p["gated_w"], pre)[0]
    tref.assert_within(dh, *back["dx"], "gated dx")
    for k, n in (("gated_w", "dweight"), ("gated_b", "dbias")):
        tref.assert_within(grads[k], *back[n], k)
    back = ref.layer_norm_backward(dh, x, mean, rstd, p["norm_w"], dy)
    for t, n in ((dx, "dx"), (grads["norm_w"], "dweight"), (grads["norm_b"], "dbias")):
        tref.assert_within(t, *back[n], n)
    assert torch.equal(grads["down_w"], dw) and torch.equal(grads["down_b"], db)


def test_single_tokens_equal_the_batch(lbp):
    """Serving one row at a time: the same numbers as the batch within both calls' bounds."""
    params = parameters(128, 300, torch.bfloat16, 7)
    x = torch.randn(20, 128, device="cuda").bfloat16()
    block = Block(lbp, params, 0.0, 1)
    h = lbp.layer_norm(x, params["norm_w"], params["norm_b"])
    assert torch.equal(h, torch.cat([lbp.layer_norm(x[i:i + 1], params["norm_w"], params["norm_b"]) for i in range(20)]))
    bound = ref.gated(h, params["gated_w"], params["gated_b"], "silu")["y"]
    rows = torch.cat([lbp.gated_linear(h[i:i + 1], params["gated_w"], params["gated_b"]) for i in range(20)])
    tref.assert_within(rows, *bound, "single rows")
    y, _ = block.forward(x, 0)
    assert y.shape == x.shape and torch.isfinite(y).all()


def test_training_step_captured(lbp):
    """A whole step (forward, backward, update, the mask's step counted up) captured and replayed
    equals the eager steps bit for bit."""
    def setup():
        params = parameters(64, 96, torch.float32, 8)
        x, t = torch.ones(50, 64, device="cuda"), torch.zeros(50, 64, device="cuda")
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        x.normal_(generator=g)
        t.normal_(generator=g)
        return params, x, t, torch.zeros(1, dtype=torch.int64, device="cuda")

    def one(params, x, t, step):
        p = params
        h, mean, rstd = lbp.layer_norm(x, p["norm_w"], p["norm_b"], want_stats=True)
        a, pre = lbp.gated_linear(h, p["gated_w"], p["gated_b"], want_pre=True)
        o = lbp.linear(a, p["down_w"], p["down_b"])
        y = lbp.dropout(o, 0.1, 3, 0, residual=x, step=step)
        dy = (y - t) / 50
        do = lbp.dropout(dy, 0.1, 3, 0, step=step)
        da, dw, db, _ = lbp.linear_backward(do, a, p["down_w"])
        dh, gw, gb = lbp.gated_linear_backward(da, h, p["gated_w"], pre)
        _, nw, nb = lbp.layer_norm_backward(dh, x, mean, rstd, p["norm_w"], want_x=False)
        for k, v in dict(norm_w=nw, norm_b=nb, gated_w=gw, gated_b=gb, down_w=dw, down_b=db).items():
            p[k].add_(v, alpha=-0.05)
        step.add_(1)

    eager, graphed = setup(), setup()
    one(*setup())                                   # everything is loaded before the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        one(*graphed)
    for k in range(4):
        one(*eager)
        graph.replay()
        torch.cuda.synchronize()
        for name in eager[0]:
            assert torch.equal(eager[0][name], graphed[0][name]), (k, name)
