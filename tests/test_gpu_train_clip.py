"""The global gradient norm and clipping against float64."""
import math

import pytest
import torch

import train_reference as ref
from helpers import ensure_built

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
LISTS = {
    "one": [(1,)], "mlp": [(100, 784), (100,), (100, 100), (100,), (10, 100), (10,)],
    "odd": [(3,), (0,), (16385,), (1, 7), (255,), (50001,), (2, 3, 5)],
    "many": [(17 + i,) for i in range(300)], "large": [(1025, 2049), (5,), (300000,)],
    "chunks": [(16384,), (16383,), (32768,), (65537,), (8,)],
}


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def make(shapes, dtypes, seed=0, std=0.02):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(*s, generator=g, device="cuda") * std).to(dtypes[i % len(dtypes)])
            for i, s in enumerate(shapes)]


def norm64(grads):
    return math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in grads))


def check(lbp, grads, max_norm, what, out=None, **kw):
    before = [g.clone() for g in grads]
    want = norm64(before)
    norm, got = lbp.clip_grad_norm(grads, max_norm, out=out, **kw)
    # float64 sums; the square root and the result are rounded once
    assert abs(float(norm) - want) <= 2 * ref.U32 * want, (what, float(norm), want)
    s = max_norm / want if want > max_norm else 1.0
    for i, (g, b) in enumerate(zip(got, before)):
        v = b.double() * s
        dt = b.dtype
        bound = 4 * ref.U32 * v.abs()
        ref.assert_within(g, v, 0.0 if s == 1.0 else bound + ref.UNIT[dt] * (v.abs() + bound) + ref.TINY[dt],
                          f"{what} tensor {i}")
    return norm, got


@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F16,), (F32, BF16, F16)], ids=str)
@pytest.mark.parametrize("name", list(LISTS))
def test_norm_and_clipping(lbp, name, dtypes):
    print(f"clip {name} {dtypes}", flush=True)
    for max_norm in (1e-3, 1e6, math.inf, 0.0):
        grads = make(LISTS[name], dtypes)
        out = [torch.empty_like(g) for g in grads]
        keep = [g.clone() for g in grads]
        n1, _ = check(lbp, grads, max_norm, f"{name} apart", out=out)
        assert all(torch.equal(a, b) for a, b in zip(grads, keep))
        n2, got = check(lbp, grads, max_norm, f"{name} in place")
        assert torch.equal(n1, n2) and all(a is b for a, b in zip(got, grads))
        assert all(torch.equal(a, b) for a, b in zip(grads, out))


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_unaligned_tensors_leave_their_surroundings(lbp, dtype):
    base = make([(100000,)], (dtype,))[0]
    for shift, n in ((1, 4095), (3, 70001), (8, 17), (5, 1)):
        buf = base.clone()
        view = buf[shift:shift + n]
        aside = torch.full_like(buf, 7.0)
        print(f"unaligned {shift} {n} {dtype}", flush=True)
        check(lbp, [view], 1e-3, "unaligned", out=[aside[shift + 1:shift + 1 + n]])
        check(lbp, [view], 1e-3, "unaligned")
        assert torch.equal(view, aside[shift + 1:shift + 1 + n])
        assert torch.equal(buf[:shift], base[:shift]) and torch.equal(buf[shift + n:], base[shift + n:])
        assert (aside[:shift + 1] == 7.0).all() and (aside[shift + 1 + n:] == 7.0).all()


def test_range_of_the_squares(lbp):
    """Squares beyond float32's range on either side."""
    for v in (1e30, 3e-38, 1e-22):
        check(lbp, [torch.full((1000,), v, device="cuda")], v, f"values {v}")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_norm_that_is_not_finite_clips_nothing(lbp, bad):
    grads = make(LISTS["odd"], (F32, F16))
    grads[5][40000] = bad
    keep = [g.clone() for g in grads]
    out = [torch.zeros_like(g) for g in grads]
    norm, _ = lbp.clip_grad_norm(grads, 0.1, out=out)
    norm2, _ = lbp.clip_grad_norm(grads, 0.1)
    for n in (norm, norm2):
        assert torch.isnan(n).all() if math.isnan(bad) else float(n) == math.inf
    for a, b, c in zip(grads, keep, out):
        assert torch.equal(a.nan_to_num(1.5), b.nan_to_num(1.5)) and torch.equal(c.nan_to_num(1.5), b.nan_to_num(1.5))
    # a norm beyond float32 is infinite as well
    big = [torch.full((100,), 3e38, device="cuda")]
    norm, _ = lbp.clip_grad_norm(big, 1.0)
    assert float(norm) == math.inf and (big[0] == torch.full_like(big[0], 3e38)).all()


def test_no_tensors_and_zeros(lbp):
    norm, out = lbp.clip_grad_norm([], 1.0)
    assert float(norm) == 0 and out == []
    z = [torch.zeros(1000, device="cuda"), torch.zeros(0, device="cuda")]
    norm, _ = lbp.clip_grad_norm(z, 0.0)
    assert float(norm) == 0 and (z[0] == 0).all()


def test_stream_graph_and_repeats(lbp):
    grads = make(LISTS["mlp"], (F32,))
    out = [torch.empty_like(g) for g in grads]
    ws = lbp.clip_grad_norm_workspace(grads)
    ws.fill_(255)
    first, _ = lbp.clip_grad_norm(grads, 0.1, out=out, ws=ws)
    keep = [o.clone() for o in out]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again, _ = lbp.clip_grad_norm(grads, 0.1, out=out, ws=ws)
    s.synchronize()
    assert torch.equal(first, again) and all(torch.equal(a, b) for a, b in zip(out, keep))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, _ = lbp.clip_grad_norm(grads, 0.1, out=out, ws=ws)
    for i in range(3):
        for g, n in zip(grads, make(LISTS["mlp"], (F32,), seed=5 + i)):
            g.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want, res = lbp.clip_grad_norm(grads, 0.1, out=[torch.empty_like(g) for g in grads])
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(got, res)), i


def test_refusals_of_the_binding(lbp):
    """Wrong tensors are refused before anything runs."""
    g = make([(4, 5), (7,)], (F32,))
    for grads, out, text in (
            ([g[0].t(), g[1]], None, "contiguous"), ([g[0], g[1].cpu()], None, "one device"),
            ([g[0].double()], None, "float32, bfloat16 or float16"), (g, [g[0]], "1 outputs for 2"),
            (g, [g[0], g[1].to(BF16)], "types"), (g, [g[0], torch.zeros(8, device="cuda")], "numbers of elements"),
            (g, [g[0], torch.zeros(7)], "one device")):
        with pytest.raises(ValueError, match=text):
            lbp.clip_grad_norm(grads, 1.0, out=out)
    with pytest.raises(lbp.VBError, match="max_norm"):
        lbp.clip_grad_norm(g, -1.0)
    with pytest.raises(lbp.VBError, match="workspace too small"):
        lbp.clip_grad_norm(g, 1.0, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
