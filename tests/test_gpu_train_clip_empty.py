"""Clipping of long lists of empty tensors: the norm is written whatever the list holds."""
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


@pytest.mark.parametrize("n", [1, 16, 17, 112, 113, 300, 1000])
def test_norm_of_empty_tensors_is_written(lbp, n):
    print(f"empty {n}", flush=True)
    grads = [torch.empty(0, device="cuda") for _ in range(n)]
    # memory that the norm may come from holds other values
    used = [torch.full((64,), 7.0, device="cuda") for _ in range(32)]
    del used
    norm, out = lbp.clip_grad_norm(grads, 1.0)
    assert float(norm) == 0.0 and len(out) == n
    norm, _ = lbp.clip_grad_norm(grads, 1.0, out=[torch.empty(0, device="cuda") for _ in range(n)])
    assert float(norm) == 0.0
    # the C call writes the caller's number
    from array import array
    from linear_bound_propagation_amd import train
    own = torch.full((1,), 7.0, device="cuda")
    ws = lbp.clip_grad_norm_workspace(grads)
    sizes, types, ptrs = array("q", [0] * n), array("i", [0] * n), array("Q", [0] * n)
    train._run("vb_clip_grad_norm", n, ptrs.buffer_info()[0], None, sizes.buffer_info()[0], types.buffer_info()[0], 1.0,
               own.data_ptr(), ws.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert float(own) == 0.0


@pytest.mark.parametrize("numbers", [1, 500, 40000])
@pytest.mark.parametrize("n, at", [(113, 112), (300, 0), (300, 150), (1000, 999)])
def test_one_tensor_among_empty_ones(lbp, n, at, numbers):
    grads = [torch.empty(0, device="cuda") for _ in range(n)]
    grads[at] = torch.full((numbers,), 3.0, device="cuda")
    norm, out = lbp.clip_grad_norm(grads, 1.5)
    want = 3.0 * numbers ** 0.5
    assert abs(float(norm) - want) <= 2.0 ** -22 * want
    assert torch.allclose(out[at], torch.full_like(out[at], 1.5 / numbers ** 0.5), rtol=2.0 ** -21, atol=0)
