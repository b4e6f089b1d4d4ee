"""Tensors that require grad: no graph is recorded, so they are refused unless none is wanted."""
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def leaf(*shape):
    return torch.randn(*shape, device="cuda", requires_grad=True)


def calls(lbp):
    """name -> (call of one tensor, shape of the tensor that requires grad)"""
    x, w, dy = torch.randn(6, 8, device="cuda"), torch.randn(5, 8, device="cuda"), torch.randn(6, 5, device="cuda")
    y = torch.zeros(6, dtype=torch.int64, device="cuda")
    return {"linear x": (lambda t: lbp.linear(t, w), (6, 8)), "linear weight": (lambda t: lbp.linear(x, t), (5, 8)),
            "linear bias": (lambda t: lbp.linear(x, w, t), (5,)), "linear residual": (lambda t: lbp.linear(x, w, None, t), (6, 5)),
            "linear out": (lambda t: lbp.linear(x, w, out=t), (6, 5)),
            "backward dy": (lambda t: lbp.linear_backward(t, x, w), (6, 5)),
            "backward x": (lambda t: lbp.linear_backward(dy, t, w), (6, 8)),
            "backward weight": (lambda t: lbp.linear_backward(dy, x, t), (5, 8)),
            "backward saved": (lambda t: lbp.linear_backward(dy, x, w, act="relu", saved=t), (6, 5)),
            "loss": (lambda t: lbp.cross_entropy(t, y), (6, 9)),
            "loss gradient": (lambda t: lbp.cross_entropy(torch.zeros(6, 9, device="cuda"), y, dlogits=t), (6, 9)),
            "clip": (lambda t: lbp.clip_grad_norm([t], 1.0), (40,)),
            "clip out": (lambda t: lbp.clip_grad_norm([torch.ones(40, device="cuda")], 1.0, out=[t]), (40,))}


@pytest.mark.parametrize("name", ["linear x", "linear weight", "linear bias", "linear residual", "linear out", "backward dy",
                                  "backward x", "backward weight", "backward saved", "loss", "loss gradient", "clip", "clip out"])
def test_refused_while_a_graph_is_recorded(lbp, name):
    call, shape = calls(lbp)[name]
    t = leaf(*shape)
    before = t.detach().clone()
    with pytest.raises(ValueError, match="no autograd graph"):
        call(t)
    assert torch.equal(t.detach(), before)
    with torch.no_grad():
        call(t)
    with torch.inference_mode():
        call(leaf(*shape))
    call(before)
    call(leaf(*shape).detach())
