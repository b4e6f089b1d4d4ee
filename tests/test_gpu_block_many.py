"""Layer norm and the gated linear layer with more rows than one dimension of a launch holds, and
calls of several streams at once."""
import pytest
import torch

import block_reference as ref
from helpers import ensure_built
from train_reference import assert_within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def small_integers(seed, *shape, most=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).half()


@pytest.mark.parametrize("n", [8, 3])
def test_norm_of_many_rows(lbp, n):
    """2^27 rows and some, 16 to a workgroup (a wavefront's quarter each)."""
    rows = 2 ** 27 + 5
    print(f"norm {rows} x {n}", flush=True)
    x, dy = small_integers(1, rows, n, most=9), small_integers(2, rows, n, most=2)
    w = torch.tensor([1.0, 2.0, 0.5, 1.0, 1.5, 1.0, 3.0, 1.0], device="cuda").half()[:n].contiguous()
    y, mean, rstd = lbp.layer_norm(x, w, w, want_stats=True)
    dx, dw, db = lbp.layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    eps = float(torch.tensor(1e-5))
    sums, bound = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 2 ** 23):
        part = slice(a, a + 2 ** 23)
        want = ref.layer_norm(x[part], w, w, eps)
        assert_within(y[part], *want["y"], f"y {a}")
        assert_within(mean[part], *want["mean"], f"mean {a}")
        back = ref.layer_norm_backward(dy[part], x[part], mean[part], rstd[part], w, None)
        assert_within(dx[part], *back["dx"], f"dx {a}")
        sums += back["dweight"][0]
        xh = (x[part].double() - mean[part].double()[:, None]) * rstd[part].double()[:, None]
        bound += (dy[part].double() * xh).abs().sum(0)
    # sums of 2^27 terms in at least 256 parts of 2^19 rows or less each: 2^20 2^-24 of the magnitudes
    assert_within(dw, sums, 2.0 ** -4 * bound + 2.0 ** -11 * sums.abs(), "dweight")
    assert torch.equal(db, dy.double().sum(0).half())


def test_gated_of_many_rows(lbp):
    """Small integers, whose sums are exact."""
    rows, n = 2 ** 27 + 70, 8
    print(f"gated {rows} x {n} -> {n}", flush=True)
    x, dy, w, pre = small_integers(3, rows, n), small_integers(4, rows, n), small_integers(5, 2 * n, n, most=2), \
        small_integers(6, rows, 2 * n)
    y = lbp.gated_linear(x, w, act="relu")
    dx, dw, db = lbp.gated_linear_backward(dy, x, w, pre, act="none")
    torch.cuda.synchronize()
    sums, products = torch.zeros(2 * n, dtype=torch.float64, device="cuda"), torch.zeros(2 * n, n, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 2 ** 23):
        part = slice(a, a + 2 ** 23)
        v = torch.mm(x[part].float(), w.float().t().contiguous())
        assert torch.equal(y[part], (v[:, :n].clamp_min(0) * v[:, n:]).half()), a
        d = dy[part].float()
        g = torch.cat([d * pre[part, n:].float(), d * pre[part, :n].float()], 1)
        assert torch.equal(dx[part], torch.mm(g, w.float()).half()), a
        sums += g.double().sum(0)
        products += torch.mm(g.double().t().contiguous(), x[part].double())
    assert torch.equal(db, sums.half()) and torch.equal(dw, products.half())


def test_calls_on_two_streams_at_once(lbp):
    """Each call with a workspace of its own gives what it gives alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda").bfloat16()

    x, w, dy, pre, gain = normal(700, 520), normal(2 * 900, 520), normal(700, 900), normal(700, 1800), normal(520)
    _, mean, rstd = lbp.layer_norm(x, gain, want_stats=True)

    def work():
        return [*lbp.gated_linear_backward(dy, x, w, pre), lbp.gated_linear(x, w), *lbp.layer_norm_backward(x, x, mean, rstd, gain),
                lbp.dropout(x, 0.3, 5, residual=x)]

    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for k, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(work())
    torch.cuda.synchronize()
    for runs in got:
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, want))
