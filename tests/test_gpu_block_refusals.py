"""The binding of the gated linear layer, layer norm and dropout refuses tensors that do not fit
each other, and those that require grad while a graph is recorded."""
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def t(*shape, dtype=torch.float32, device="cuda"):
    return torch.ones(*shape, dtype=dtype, device=device)


def test_wrong_tensors(lbp):
    x, w, b, dy, pre, s = t(6, 8), t(10, 8), t(10), t(6, 5), t(6, 10), t(6)
    h = torch.float16
    for text, call in (
            ("matrix", lambda: lbp.gated_linear(t(6), w)), ("matrix", lambda: lbp.gated_linear(x, t(9, 8))),
            ("matrix", lambda: lbp.gated_linear(x, t(10))), ("weight must be", lambda: lbp.gated_linear(x, t(10, 7))),
            ("weight must be", lambda: lbp.gated_linear(x, t(10, 8, dtype=h))), ("bias must be", lambda: lbp.gated_linear(x, w, t(5))),
            ("act must be", lambda: lbp.gated_linear(x, w, act="tanh")), ("out must be", lambda: lbp.gated_linear(x, w, out=t(6, 10))),
            ("float32, bfloat16", lambda: lbp.gated_linear(x.double(), w.double())), ("contiguous", lambda: lbp.gated_linear(t(8, 6).t(), w)),
            ("dy must be", lambda: lbp.gated_linear_backward(pre, x, w, pre)), ("pre must be", lambda: lbp.gated_linear_backward(dy, x, w, dy)),
            ("current GPU", lambda: lbp.gated_linear(x.cpu(), w)), ("weight must be", lambda: lbp.gated_linear(x, w.cpu())),
            ("weight must be", lambda: lbp.layer_norm(x, t(7))), ("bias must be", lambda: lbp.layer_norm(x, None, t(8, 1))),
            ("out must be", lambda: lbp.layer_norm(x, out=t(6, 9))), ("matrix", lambda: lbp.layer_norm(t(8))),
            ("dy must be", lambda: lbp.layer_norm_backward(t(6, 7), x, s, s)), ("mean must be", lambda: lbp.layer_norm_backward(x, x, s.half(), s)),
            ("rstd must be", lambda: lbp.layer_norm_backward(x, x, s, t(7))), ("dresidual must be", lambda: lbp.layer_norm_backward(x, x, s, s, dresidual=t(5, 8))),
            ("dx must be", lambda: lbp.layer_norm_backward(x, x, s, s, dx=t(6, 9))), ("ws must be", lambda: lbp.layer_norm_backward(x, x, s, s, ws=t(4096, device="cpu"))),
            ("seed and offset", lambda: lbp.dropout(x, 0.5, -1)), ("seed and offset", lambda: lbp.dropout(x, 0.5, 1, 2 ** 64)),
            ("residual must be", lambda: lbp.dropout(x, 0.5, 1, residual=t(6, 7))), ("step must be", lambda: lbp.dropout(x, 0.5, 1, step=s[:1])),
            ("out must be", lambda: lbp.dropout(x, 0.5, 1, out=x.half())), ("matrix", lambda: lbp.dropout(t(5), 0.5, 1))):
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(lbp.VBError, match="p must"):
        lbp.dropout(x, 1.5, 1)
    with pytest.raises(lbp.VBError, match="eps"):
        lbp.layer_norm(x, eps=-1.0)
    with pytest.raises(lbp.VBError, match="overlaps"):
        lbp.gated_linear(x, t(16, 8), out=x)
    with pytest.raises(lbp.VBError, match="overlaps"):
        lbp.dropout(x[1:], 0.5, 1, out=x[:-1])


def test_no_graph(lbp):
    x, w, dy, pre, s = t(6, 8), t(10, 8), t(6, 5), t(6, 10), t(6)
    calls = [(lambda a: lbp.gated_linear(a, w), (6, 8)), (lambda a: lbp.gated_linear(x, a), (10, 8)),
             (lambda a: lbp.gated_linear(x, w, a), (10,)), (lambda a: lbp.gated_linear_backward(a, x, w, pre), (6, 5)),
             (lambda a: lbp.gated_linear_backward(dy, x, a, pre), (10, 8)), (lambda a: lbp.gated_linear_backward(dy, x, w, a), (6, 10)),
             (lambda a: lbp.layer_norm(a), (6, 8)), (lambda a: lbp.layer_norm(x, a), (8,)), (lambda a: lbp.layer_norm(x, None, a), (8,)),
             (lambda a: lbp.layer_norm_backward(a, x, s, s), (6, 8)), (lambda a: lbp.layer_norm_backward(x, x, s, s, a), (8,)),
             (lambda a: lbp.layer_norm_backward(x, x, s, s, dresidual=a), (6, 8)), (lambda a: lbp.dropout(a, 0.5, 1), (6, 8)),
             (lambda a: lbp.dropout(x, 0.5, 1, residual=a), (6, 8)), (lambda a: lbp.dropout(x, 0.5, 1, out=a), (6, 8))]
    for i, (call, shape) in enumerate(calls):
        leaf = torch.randn(*shape, device="cuda", requires_grad=True)
        before = leaf.detach().clone()
        with pytest.raises(ValueError, match="no autograd graph"):
            call(leaf)
        assert torch.equal(leaf.detach(), before), i
        with torch.no_grad():
            call(leaf.detach().clone().requires_grad_())
        call(before)
