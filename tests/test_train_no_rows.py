"""The backward pass without rows: dx and dresidual are empty, and an empty tensor's address is
NULL, so a call that wants nothing else has nothing to do and is none to refuse."""
import ctypes

import pytest

from helpers import ensure_built

ensure_built()
import linear_bound_propagation_amd as lbp  # noqa: E402
from linear_bound_propagation_amd import train  # noqa: E402

L = lbp.lib()


@pytest.mark.parametrize("act", [0, 1, 2, 3])
def test_only_empty_gradients(act):
    p = train.vb_linear_bwd(rows=0, n_in=12, n_out=10, dtype=1, act=act, ld_dy=10, ld_x=12, weight=4096, ld_w=12, ld_saved=10,
                            ld_dx=12, ld_dres=10)
    assert L.vb_linear_backward(ctypes.byref(p), None, 0, None) == 0
    p.rows = 1
    assert L.vb_linear_backward(ctypes.byref(p), None, 0, None) == -1
