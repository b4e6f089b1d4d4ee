"""float16: the range of the gradient of pre, as an operand of the gated layer's backward products."""
import pytest
import torch

import block_reference as ref
from helpers import ensure_built
from train_reference import assert_within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def make(rows, n_in, n_out):
    """Positive weights and inputs; without an activation g = (dy * up | dy * gate), small everywhere."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def uniform(*s, low, high):
        return (low + (high - low) * torch.rand(*s, generator=g, device="cuda")).half()

    return uniform(rows, n_in, low=0.5, high=1), uniform(2 * n_out, n_in, low=2.0 ** -9, high=2.0 ** -8), \
        uniform(rows, n_out, low=-1, high=1), uniform(rows, 2 * n_out, low=-1, high=1)


@pytest.mark.parametrize("size", [(3, 8, 4), (70, 130, 33), (300, 64, 515)], ids=str)
def test_range_of_g(lbp, size):
    rows, n_in, n_out = size
    x, w, dy, pre = make(*size)
    dy[0, 1], pre[0, n_out + 1] = 500.0, 1.0
    clean = lbp.gated_linear_backward(dy, x, w, pre, act="none")
    clean_one = lbp.gated_linear_backward(dy, x, w, pre, act="none", round_g=True)
    # g = 500 * up of row 0, output 1
    for up, one, two in ((131.0, True, True), (140.0, False, True), (262.0, False, True), (263.0, False, False)):
        print(f"{size} g {500 * up}", flush=True)
        p = pre.clone()
        p[0, n_out + 1] = up
        for round_g, finite, base in ((True, one, clean_one), (False, two, clean)):
            dx, dw, db = lbp.gated_linear_backward(dy, x, w, p, act="none", round_g=round_g)
            if finite:
                want = ref.gated_backward(dy, x, w, p, "none", round_g)
                assert_within(dx, *want["dx"], f"dx {up}")
                # dweight of that row may pass float16's largest number
                ok = (want["dweight"][0].abs() < 65000).all(1)
                assert_within(dw[ok], want["dweight"][0][ok], want["dweight"][1][ok], f"dweight {up}")
            else:
                assert torch.isposinf(dx[0]).all() and torch.isposinf(dw[1]).all()
            # other rows of dx and of dweight have nothing of it
            assert torch.equal(dx[1:], base[0][1:])
            others = torch.arange(2 * n_out, device="cuda") != 1
            assert torch.equal(dw[others], base[1][others]) and torch.equal(db[others], base[2][others])


def test_dbias_sums_float32_numbers(lbp):
    """g beyond the products' range that cancels in the sum: 150000 - 130000 is a float16 number."""
    x, w, dy, pre = make(2, 8, 4)
    dy[:, 1], pre[0, 5], pre[1, 5] = 500.0, 300.0, -260.0
    for round_g in (False, True):
        db = lbp.gated_linear_backward(dy, x, w, pre, act="none", round_g=round_g)[2]
        assert float(db[1]) == 20000.0
    up = pre[:, 4:].double()
    assert float((dy.double() * up).sum(0)[1]) == 20000.0
