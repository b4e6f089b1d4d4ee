"""Host checks of the choice between one and two 16-bit numbers for the gradient of the
pre-activation (fake device addresses: nothing is dereferenced)."""
import ctypes

import pytest

from helpers import ensure_built

ensure_built()
import linear_bound_propagation_amd as lbp  # noqa: E402
from linear_bound_propagation_amd import train  # noqa: E402

L = lbp.lib()


def args(**kw):
    d = dict(rows=500, n_in=64, n_out=40, dtype=1, act=2, dy=4096, ld_dy=40, x=4096, ld_x=64, weight=8192, ld_w=64,
             saved=16384, ld_saved=40, dx=1 << 20, ld_dx=64, dweight=1 << 21, ld_dw=64)
    d.update(kw)
    return ctypes.byref(train.vb_linear_bwd(**d))


def need(**kw):
    out = ctypes.c_size_t(0)
    assert L.vb_linear_backward_workspace(args(**kw), ctypes.byref(out)) == 0
    return out.value


def test_workspace_holds_two_numbers_unless_rounded():
    one = 500 * 40 * 2
    for act in (2, 3):
        for dtype in (1, 2):
            assert need(act=act, dtype=dtype) >= 2 * one
            assert one <= need(act=act, dtype=dtype, round_g=1) < 2 * one
        assert need(act=act, dtype=0, ld_dy=40) == need(act=act, dtype=0, round_g=1)
    assert need(act=1) == need(act=1, round_g=1) and need(act=0) == need(act=0, round_g=1)


@pytest.mark.parametrize("bad", [-1, 2])
def test_refusal(bad):
    assert L.vb_linear_backward(args(round_g=bad), None, 0, None) == -1
    assert "round_g" in L.vb_last_error().decode()
