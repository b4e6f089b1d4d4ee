"""Outputs that share memory with another argument are refused; rows that lie between each
other's are not, and give the same results."""
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def normal(*shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda").to(dtype)


def test_refused(lbp):
    x, w = normal(40, 30), normal(30, 30)
    z, y = normal(20, 33), torch.zeros(20, dtype=torch.int64, device="cuda")
    grads = [normal(50), normal(50)]
    keep = [t.clone() for t in (x, w, z, *grads)]
    for call in (lambda: lbp.linear(x, w, out=x), lambda: lbp.linear(x[:30], w, out=w),
                 lambda: lbp.linear(x[1:], w, residual=x[:-1], out=x[:-1]), lambda: lbp.linear(w, w, out=w),
                 lambda: lbp.cross_entropy(z[:, :-1], y, dlogits=z[:, 1:]),
                 lambda: lbp.clip_grad_norm(grads, 0.1, out=grads[::-1]), lambda: lbp.clip_grad_norm(grads + grads[:1], 0.1),
                 lambda: lbp.linear(x, w, ws=x)):
        try:
            call()
        except lbp.VBError as e:
            assert "overlap" in str(e) or "workspace too small" in str(e), e
        else:
            # a workspace that the call does not use may be anything
            assert torch.equal(x, keep[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((x, w, z, *grads), keep))
    for call in (lambda: lbp.linear(x, w, out=x), lambda: lbp.cross_entropy(z[:, :-1], y, dlogits=z[:, 1:]),
                 lambda: lbp.clip_grad_norm(grads, 0.1, out=grads[::-1])):
        with pytest.raises(lbp.VBError, match="overlap"):
            call()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16], ids=str)
def test_columns_of_one_buffer(lbp, dtype):
    """Input, residual and output as column ranges of one buffer; logits and gradient too."""
    rows, n_in, n_out = 70, 40, 24
    buf = normal(rows, n_in + 2 * n_out, dtype=dtype)
    x, r, out = buf[:, :n_in], buf[:, n_in:n_in + n_out], buf[:, n_in + n_out:]
    w = normal(n_out, n_in, dtype=dtype)
    want = lbp.linear(x.contiguous(), w, residual=r.contiguous(), act="relu")
    assert lbp.linear(x, w, residual=r, act="relu", out=out) is out and torch.equal(out, want)
    assert torch.equal(lbp.linear(x, w, residual=r, act="relu", out=r), want)         # over the residual
    y = torch.randint(0, n_in, (rows,), device="cuda")
    grad = lbp.cross_entropy(x.contiguous(), y)[2]
    side = torch.cat([x, torch.zeros_like(x)], 1)
    assert torch.equal(lbp.cross_entropy(side[:, :n_in], y, dlogits=side[:, n_in:])[2], grad)
    assert torch.equal(lbp.cross_entropy(side[:, :n_in], y, dlogits=side[:, :n_in])[2], grad)


def test_gradients_read_twice(lbp):
    """Gradients may repeat where they are only read."""
    g = normal(1000)
    norm, out = lbp.clip_grad_norm([g, g], 0.5, out=[torch.empty_like(g), torch.empty_like(g)])
    assert torch.equal(out[0], out[1])
    assert abs(float(norm) - float((2 * (g.double() ** 2).sum()).sqrt())) <= 2.0 ** -22 * float(norm)
