"""Dropout: the mask against the generator in integers, the values against float64."""
import math

import pytest
import torch

import block_reference as ref
from helpers import ensure_built
from train_reference import assert_within

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
SIZES = [(1, 1), (1, 3), (3, 4), (5, 5), (16, 100), (7, 1001), (128, 64), (33, 2047), (2, 2056), (3, 5000), (1, 100003), (70001, 2)]


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_values(lbp, size, dtype):
    x, res = normal(1, *size, dtype=dtype), normal(2, *size, dtype=dtype)
    for p, seed, offset in ((0.1, 7, 0), (0.5, 2 ** 63 + 12345, 2 ** 33 + 5), (0.97, 2 ** 64 - 1, 2 ** 64 - 1), (2.0 ** -10, 3, 1)):
        mask = ref.kept(*size, p, seed, offset)
        for r in (None, res):
            what = f"dropout {size} {dtype} {p} {r is not None}"
            print(what, flush=True)
            y = lbp.dropout(x, p, seed, offset, residual=r)
            assert_within(y, *ref.dropout(x, p, mask, r), what)
            if r is None:
                zero = mask.to(y.device).logical_not()
                assert (y[zero] == 0).all()


def test_words_of_the_generator():
    """The numpy form of the mask is that of the integers' one, element by element."""
    mask = ref.kept(5, 11, 0.3, 2 ** 40 + 9, 2 ** 35 + 1, first_row=2 ** 33)
    for r in range(5):
        for c in range(11):
            quad = (2 ** 33 + r) * 3 + c // 4
            word = ref.philox((quad & 0xFFFFFFFF, quad >> 32, 1, 8), ((2 ** 40 + 9) & 0xFFFFFFFF, 2 ** 8))[c % 4]
            assert bool(mask[r, c]) == (word >= round(0.3 * 2 ** 32))


def test_nothing_and_everything(lbp):
    x = normal(3, 40, 50)
    x[3, 4], x[5, 6] = math.inf, math.nan
    y = lbp.dropout(x, 0.0, 1)
    assert torch.equal(y.nan_to_num(7.0, 8.0), x.nan_to_num(7.0, 8.0))
    assert (lbp.dropout(x, 1.0, 1) == 0).all()                      # also where x is no number
    r = normal(4, 40, 50)
    assert torch.equal(lbp.dropout(x, 1.0, 1, residual=r), r)
    mask = ref.kept(40, 50, 0.5, 9, 2).cuda()
    bad = torch.where(mask, x, torch.full_like(x, math.nan))
    y = lbp.dropout(bad, 0.5, 9, 2)
    assert (y[~mask] == 0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n", [1, 30, 1001, 2056])
def test_strides_in_place_and_types(lbp, n, dtype):
    """The mask depends on nothing but row, column, width, seed and offset."""
    rows = 9
    x, r = normal(5, rows, n, dtype=dtype), normal(6, rows, n, dtype=dtype)
    want = lbp.dropout(x, 0.3, 11, 4, residual=r)
    for pad, shift in ((8, 0), (5, 0), (3, 1)):
        def view(t):
            buf = torch.full((rows, n + pad), 9.0, dtype=dtype, device="cuda")
            buf[:, shift:shift + n] = t
            return buf, buf[:, shift:shift + n]

        (xb, xv), (rb, rv), (ob, ov) = view(x), view(r), view(r)
        assert lbp.dropout(xv, 0.3, 11, 4, residual=rv, out=ov) is ov and torch.equal(ov, want)
        assert torch.equal(lbp.dropout(xv, 0.3, 11, 4, residual=rv, out=rv), want)
        rb, rv = view(r)
        assert torch.equal(lbp.dropout(xv, 0.3, 11, 4, residual=rv, out=xv), want)
        for b in (xb, rb, ob):
            b[:, shift:shift + n] = 9.0
            assert (b == 9.0).all()
    ones = torch.ones(rows, n, device="cuda")
    assert torch.equal(lbp.dropout(ones, 0.3, 11, 4) > 0, lbp.dropout(ones.to(dtype), 0.3, 11, 4) > 0)
    both = normal(7, rows, n, dtype=dtype)
    want = lbp.dropout(both.clone(), 0.3, 1, residual=both.clone())
    assert torch.equal(lbp.dropout(both, 0.3, 1, residual=both, out=both), want)


def test_shares_and_independence(lbp):
    """Shares of kept elements of 2^22, and of pairs in neighbouring places, rows, offsets and seeds:
    within six standard deviations of the binomial's."""
    rows, n = 2048, 2048
    ones = torch.ones(rows, n, device="cuda")
    total = rows * n
    for p in (0.1, 0.5, 0.9):
        a = lbp.dropout(ones, p, 42, 0) > 0
        q = 1 - p

        def near(share, expect, count):
            return abs(share - expect) <= 6 * math.sqrt(expect * (1 - expect) / count)

        assert near(float(a.double().mean()), q, total)
        for b in (lbp.dropout(ones, p, 42, 1) > 0, lbp.dropout(ones, p, 43, 0) > 0, a.roll(1, 0), a.roll(1, 1), a.roll(4, 1)):
            assert near(float((a & b).double().mean()), q * q, total)


def test_rows_past_32_bits(lbp):
    """Counters past 2^32: 2^27 + 3 rows of 130 columns take 33 each."""
    rows, n = 2 ** 27 + 3, 130
    x = torch.ones(1, n, dtype=torch.float16, device="cuda").expand(rows, n)
    print("dropout of many rows", flush=True)
    with pytest.raises(lbp.VBError, match="leading dimension"):
        lbp.dropout(x, 0.5, 5)                          # rows on top of each other
    x = torch.ones(rows, n, dtype=torch.float16, device="cuda")
    y = lbp.dropout(x, 0.5, 5, 1, out=x)
    torch.cuda.synchronize()
    for first in (0, 2 ** 27 - 50000, rows - 64):
        assert torch.equal(y[first:first + 64].cpu() > 0, ref.kept(64, n, 0.5, 5, 1, first_row=first))


def test_no_rows(lbp):
    x = torch.empty(0, 50, device="cuda")
    assert lbp.dropout(x, 0.5, 1).shape == (0, 50)
    assert lbp.dropout(x, 0.5, 1, residual=x).shape == (0, 50)


def test_captured_steps(lbp):
    """A captured call takes another mask each time its step has moved on, the backward one the same."""
    x, dy = normal(8, 200, 300, dtype=torch.bfloat16), normal(9, 200, 300, dtype=torch.bfloat16)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lbp.dropout(x, 0.4, 77, 10, step=step, out=y)
        lbp.dropout(dy, 0.4, 77, 10, step=step, out=dx)
        step.add_(1)
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        kept = [y.clone(), dx.clone()]
        assert torch.equal(kept[0], lbp.dropout(x, 0.4, 77, 10 + k)), k
        assert torch.equal(kept[1], lbp.dropout(dy, 0.4, 77, 10 + k)), k
        torch.cuda.synchronize()
    # modulo 2^64
    step.fill_(-3)
    assert torch.equal(lbp.dropout(x, 0.4, 77, 5, step=step), lbp.dropout(x, 0.4, 77, 2))
    assert torch.equal(lbp.dropout(x, 0.4, 77, 1, step=step), lbp.dropout(x, 0.4, 77, 2 ** 64 - 2))
