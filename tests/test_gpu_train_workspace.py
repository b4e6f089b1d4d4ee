"""A caller's workspace has to be contiguous memory of the GPU that the call runs on: anything
else is refused before a launch."""
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def calls(lbp):
    x, w = torch.randn(40, 30, device="cuda"), torch.randn(20, 30, device="cuda")
    z, y = torch.randn(6, 9, device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda")
    g = [torch.randn(50, device="cuda")]
    return {"linear": lambda ws: lbp.linear(x, w, ws=ws),
            "linear_backward": lambda ws: lbp.linear_backward(torch.ones(40, 20, device="cuda"), x, w, ws=ws),
            "cross_entropy": lambda ws: lbp.cross_entropy(z, y, ws=ws),
            "clip_grad_norm": lambda ws: lbp.clip_grad_norm(g, 1.0, ws=ws)}


@pytest.mark.parametrize("name", ["linear", "linear_backward", "cross_entropy", "clip_grad_norm"])
def test_workspace_elsewhere_is_refused(lbp, name):
    call = calls(lbp)[name]
    size = 1 << 20
    for bad in (torch.empty(size, dtype=torch.uint8), torch.empty(size, dtype=torch.uint8).pin_memory(),
                torch.empty(2 * size, dtype=torch.uint8, device="cuda")[::2],
                torch.empty(1, dtype=torch.uint8, device="cuda").expand(size),
                torch.empty(size // 4, 4, device="cuda").t()):
        with pytest.raises(ValueError, match="ws must be contiguous"):
            call(bad)
    call(torch.empty(size, dtype=torch.uint8, device="cuda"))
    call(torch.empty(size // 4, device="cuda"))         # of any type
