"""dweight and dbias of layer norm over very many rows."""
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu

ROWS = 2 ** 27 + 5


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def test_short_rows_keep_their_bits(lbp):
    """Rows of less than 16 bytes, all numbers equal, so that roundings do not cancel: a thread adds
    ROWS / 2^18 < 514 rows, 256 of those sums make a part's, 64 parts a thread's and 16 threads the
    result: 850 additions, each off by 2^-24 of a sum that is no larger than the result, and 2^-24 for the
    product and the last rounding each."""
    print("equal rows", flush=True)
    dy = torch.full((ROWS, 3), 0.1, device="cuda")
    x = torch.full((ROWS, 3), 3.0, device="cuda")
    mean, rstd = torch.zeros(ROWS, device="cuda"), torch.ones(ROWS, device="cuda")
    _, dw, db = lbp.layer_norm_backward(dy, x, mean, rstd, want_x=False)
    one = float(dy[0, 0])
    for got, want in ((dw, 3 * one * ROWS), (db, one * ROWS)):
        assert float((got.double() - want).abs().max()) <= 852 * 2.0 ** -24 * want
