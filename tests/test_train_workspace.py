"""The binding's check of a caller's workspace."""
import pytest
import torch

from helpers import ensure_built

ensure_built()
from linear_bound_propagation_amd import train  # noqa: E402


def test_host_and_strided_workspaces_are_refused():
    for bad in (torch.empty(4096, dtype=torch.uint8), torch.empty(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws must be contiguous on the current GPU"):
            train._scratch(bad, 0)
    own = torch.empty(4096, dtype=torch.float32)        # device -1: the host's own
    assert train._scratch(own, -1) == (own.data_ptr(), 4 * 4096)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        train._scratch(own[::2], -1)


def test_workspaces_are_not_made_for_host_tensors():
    for call in (lambda: train.linear_workspace(torch.zeros(4, 3), torch.zeros(5, 3)),
                 lambda: train.cross_entropy_workspace(torch.zeros(4, 3)),
                 lambda: train.clip_grad_norm_workspace([torch.zeros(4)])):
        with pytest.raises(ValueError, match="current GPU"):
            call()
