"""The backward pass without rows gives every combination of gradients."""
import itertools

import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
def test_each_combination(lbp, act, dtype):
    x, w = torch.empty(0, 12, dtype=dtype, device="cuda"), torch.ones(10, 12, dtype=dtype, device="cuda")
    dy = torch.empty(0, 10, dtype=dtype, device="cuda")
    for want in itertools.product((False, True), repeat=4):
        if not any(want):
            continue
        used = [torch.full((10, 12), 7.0, dtype=dtype, device="cuda") for _ in range(8)]
        del used                        # memory that the gradients may come from holds other values
        out = lbp.linear_backward(dy, x, w, act=act, saved=None if act == "none" else dy, want_x=want[0], want_weight=want[1],
                                  want_bias=want[2], want_residual=want[3])
        for t, wanted, shape in zip(out, want, ((0, 12), (10, 12), (10,), (0, 10))):
            assert (t is not None) == wanted and (t is None or (t.shape == shape and not t.any()))
