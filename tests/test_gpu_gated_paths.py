"""The gated linear layer's few-row kernels where gate and up lie at other distances from 16-byte
boundaries, with two and four blocks of weight rows, and on either side of a split reduction."""
import pytest
import torch

import block_reference as ref
from helpers import ensure_built
from test_gpu_gated import ACTS, TYPES, make
from train_reference import assert_within

pytestmark = pytest.mark.gpu

# blocks of both halves: four with 17 .. 32 rows, two, four with other distances of both halves;
# then long rows of few weights, copied for a split reduction or read in place
SIZES = [(24, 64, 5000), (20, 131, 2501), (9, 1001, 7001), (27, 65, 7001), (32, 40, 1700), (17, 33, 6400), (16, 77, 7001),
         (5, 303, 3501), (7, 8191, 2048), (16, 8193, 301), (16, 8193, 1025), (31, 2049, 300), (31, 5001, 151), (6, 4097, 31)]


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(lbp, size, dtype):
    x, w, b, _, _ = make(*size, dtype, 21)
    for name in ACTS:
        what = f"gated {size} {dtype} {name}"
        print(what, flush=True)
        y, pre = lbp.gated_linear(x, w, b, act=name, want_pre=True)
        want = ref.gated(x, w, b, name)
        assert_within(y, *want["y"], f"{what} y")
        assert_within(pre, *want["pre"], f"{what} pre")
        assert torch.equal(lbp.gated_linear(x, w, b, act=name), y)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", [(20, 131, 2501), (9, 1001, 7001), (7, 8191, 300), (16, 4100, 1000), (31, 2049, 300)], ids=str)
def test_strides(lbp, size, dtype):
    """Rows of weights and x from any element on, their surroundings NaN; outputs inside a buffer."""
    rows, n_in, n_out = size
    x, w, b, _, _ = make(*size, dtype, 22)
    want = ref.gated(x, w, b, "silu")
    for pad, shift in ((8, 0), (5, 0), (3, 1), (1, 1)):
        def view(t):
            buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
            v = buf[:, shift:shift + t.shape[1]]
            v.copy_(t)
            return v

        print(f"gated strided {size} {dtype} {pad} {shift}", flush=True)
        buf = torch.full((rows, n_out + pad), 5.0, dtype=dtype, device="cuda")
        out = buf[:, shift:shift + n_out]
        xv, wv = view(x), view(w)
        lbp.gated_linear(xv, wv, b, out=out, ws=lbp.gated_linear_workspace(xv, wv))
        assert_within(out, *want["y"], "y")
        out.fill_(5.0)
        assert bool((buf == 5.0).all())
