"""Calls whose rows or outputs take more workgroups than one dimension of a launch holds."""
import pytest
import torch

from helpers import ensure_built

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


def test_loss_of_many_short_rows(lbp):
    """2^26 rows and some, four to a workgroup of 256 threads."""
    rows = 2 ** 26 + 5
    print(f"loss {rows} x 2", flush=True)
    z = small_integers(1, rows, 2, most=3)
    labels = torch.arange(rows, device="cuda") % 2
    labels[::7] = -100
    n = int((labels != -100).sum())
    loss, row, grad = lbp.cross_entropy(z, labels, grad_scale=float(n))
    torch.cuda.synchronize()
    d = (z[:, 0] - z[:, 1]).float()                     # exact
    d = torch.where(labels == 0, -d, d)                 # loss of two classes: log(1 + exp(other - own))
    want = torch.where(labels == -100, 0.0, torch.log1p(torch.exp(d.double())))
    assert float((row.double() - want).abs().max()) <= 2.0 ** -18 * 7
    assert abs(float(loss) - float(want.sum() / n)) <= 2.0 ** -18 * 7
    p = torch.where(labels == -100, 0.0, torch.sigmoid(d.double()))     # of the other class
    for k in (0, 1):
        own = torch.where(labels == k, -p, p)
        assert float((grad[:, k].double() - own).abs().max()) <= 2.0 ** -12 + 2.0 ** -18


def test_layer_of_many_rows(lbp):
    """2^27 rows and some: more than 2^21 tiles forward, more than 2^21 parts of the rows backward.
    Small integers, whose sums are exact."""
    rows, n = 2 ** 27 + 70, 8
    print(f"layer {rows} x {n} -> {n}", flush=True)
    x, dy, w = small_integers(2, rows, n), small_integers(3, rows, n), small_integers(4, n, n, most=2)
    y = lbp.linear(x, w, act="relu")
    torch.cuda.synchronize()
    for a in range(0, rows, 2 ** 24):
        part = slice(a, a + 2 ** 24)
        assert torch.equal(y[part], torch.mm(x[part].float(), w.float().t().contiguous()).clamp_min(0).half()), a
    dx, dw, db, _ = lbp.linear_backward(dy, x, w, act="relu", saved=y)
    torch.cuda.synchronize()
    sums, products = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, n, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 2 ** 24):
        part = slice(a, a + 2 ** 24)
        g = torch.where(y[part] > 0, dy[part].float(), torch.zeros((), device="cuda"))
        assert torch.equal(dx[part], torch.mm(g, w.float()).half()), a
        sums += g.double().sum(0)
        products += torch.mm(g.double().t().contiguous(), x[part].double())
    assert torch.equal(db, sums.half()) and torch.equal(dw, products.half())


def test_zero_gradients_of_a_large_weight(lbp):
    """No rows: 2^32 16-bit zeros and some are written."""
    n_out, n_in = 65537, 65536
    used = torch.full((n_out, n_in), 7.0, dtype=torch.float16, device="cuda")
    w = used[:, :n_in]
    empty = used[:0]
    old = torch.full((n_out, n_in), 7.0, dtype=torch.float16, device="cuda")
    del old                                             # the gradient's memory, most likely
    dw = lbp.linear_backward(torch.empty(0, n_out, dtype=torch.float16, device="cuda"), empty, w, want_x=False)[1]
    torch.cuda.synchronize()
    assert dw.shape == (n_out, n_in)
    for a in range(0, n_out, 8192):
        assert not dw[a:a + 8192].any(), a
