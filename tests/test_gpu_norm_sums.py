"""dweight and dbias of layer norm: each way that they are summed, and very many rows."""
import pytest
import torch

import block_reference as ref
from helpers import ensure_built
from test_gpu_norm import TYPES, check, make
from train_reference import assert_within

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


# either way of the sums beyond 64 rows, and the row ends of each: parts of workgroups of 512 and 1024
# threads with one and two chunks a thread, columns of rows that do and do not end on a chunk
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", [(1300, 2051), (1300, 4093), (1100, 9003), (300, 9001), (200, 40003), (256, 8192), (300, 8193),
                                  (200, 5000), (100, 6001), (600, 12000), (1500, 16381), (700, 500), (300, 1300), (65, 3), (1025, 7), (3001, 5)], ids=str)
def test_both_ways(lbp, size, dtype):
    x, w, b, dy, res = make(*size, dtype, 31)
    what = f"norm backward {size} {dtype}"
    print(what, flush=True)
    _, mean, rstd = lbp.layer_norm(x, w, b, want_stats=True)
    want = ref.layer_norm_backward(dy, x, mean, rstd, w, res)
    got = lbp.layer_norm_backward(dy, x, mean, rstd, w, dresidual=res)
    check(dict(zip(("dx", "dweight", "dbias"), got)), want, what)
    only = [lbp.layer_norm_backward(dy, x, mean, rstd, w, dresidual=res, want_x=i == 0, want_weight=i == 1, want_bias=i == 2)[i]
            for i in range(3)]
    assert all(torch.equal(a, c) for a, c in zip(only, got))
    plain = lbp.layer_norm_backward(dy, x, mean, rstd, w)
    check(dict(zip(("dx", "dweight", "dbias"), plain)), ref.layer_norm_backward(dy, x, mean, rstd, w, None), f"{what} alone")
    for over in (dy.clone(), res.clone()):                # dx over dy, over dresidual
        first = over if torch.equal(over, dy) else dy
        second = over if first is dy else res
        again = lbp.layer_norm_backward(first, x, mean, rstd, w, dresidual=second, dx=over)
        assert again[0] is over and all(torch.equal(a, c) for a, c in zip(again, got))


def small_integers(seed, *shape, most):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("n, dtype", [(8, torch.float32), (3, torch.float32), (8, torch.float16), (7, torch.bfloat16)], ids=str)
def test_exact_sums_of_many_rows(lbp, n, dtype):
    """Small integers with a mean of 0 and rstd of 1 as the statistics: the sums, and any part of them, are
    integers far below 2^24 (their standard deviation is 1.3e4), so that every row counts exactly once."""
    print(f"{ROWS} x {n} {dtype}", flush=True)
    x, dy = small_integers(1, ROWS, n, most=1), small_integers(2, ROWS, n, most=2)
    want_w, want_b = (x * dy).sum(0, dtype=torch.int64), dy.sum(0, dtype=torch.int64)
    mean, rstd = torch.zeros(ROWS, device="cuda"), torch.ones(ROWS, device="cuda")
    assert int(want_w.abs().max()) < 65504 and int(want_b.abs().max()) < 65504
    _, dw, db = lbp.layer_norm_backward(dy.to(dtype), x.to(dtype), mean, rstd, want_x=False)
    assert torch.equal(dw, want_w.double().to(dtype)) and torch.equal(db, want_b.double().to(dtype))
    _, dw, db = lbp.layer_norm_backward(dy.to(dtype), x.to(dtype), mean, rstd)
    assert torch.equal(dw, want_w.double().to(dtype)) and torch.equal(db, want_b.double().to(dtype))


@pytest.mark.parametrize("n", [8, 3])
def test_statistics_of_many_rows(lbp, n):
    x = small_integers(3, ROWS, n, most=9).half()
    _, mean, rstd = lbp.layer_norm(x, want_stats=True)
    for a in range(0, ROWS, 2 ** 23):
        part = slice(a, a + 2 ** 23)
        want = ref.layer_norm(x[part], None, None, float(torch.tensor(1e-5)))
        assert_within(mean[part], *want["mean"], f"mean {a}")
        assert_within(rstd[part], *want["rstd"], f"rstd {a}")


def test_small_spreads(lbp):
    """The float32 squares of differences of 1e-18 are normal numbers, those of 1e-24 are 0."""
    x, w, b, _, _ = make(4, 300, torch.float32, 41, mean=0.0)
    y, mean, rstd = lbp.layer_norm(x * 1e-18, w, b, eps=0.0, want_stats=True)
    check({"y": y, "mean": mean, "rstd": rstd}, ref.layer_norm(x * 1e-18, w, b, 0.0), "spread 1e-18")
    _, _, rstd = lbp.layer_norm(x * 1e-24, w, b, eps=0.0, want_stats=True)
    assert torch.isposinf(rstd).all()
    y, mean, rstd = lbp.layer_norm(x * 1e-24, w, b, want_stats=True)
    check({"y": y, "mean": mean, "rstd": rstd}, ref.layer_norm(x * 1e-24, w, b, float(torch.tensor(1e-5))), "spread 1e-24")
