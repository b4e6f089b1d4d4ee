"""GELU and SiLU and their derivatives by themselves: a layer with the weight 1 at every finite
16-bit number (and float32 numbers over the same range), against float64 with bounds relative to
the result, in the lower tail too."""
import math

import pytest
import torch

import train_reference as ref
from helpers import ensure_built

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def ndtr(v):
    """The normal CDF in float64, by erfc: torch's own is (1 + erf) / 2, with nothing left below -8."""
    return 0.5 * torch.special.erfc(v * -0.5 ** 0.5)


def numbers(dtype):
    if dtype == F32:
        v = torch.cat([torch.linspace(-14, 14, 40001), torch.linspace(-100, 100, 5001)])
    else:
        v = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(dtype)
        v = v[torch.isfinite(v)]
    return v.to(dtype).cuda()


def relative(dtype, act, v):
    """Relative error of Phi and of exp(-v^2/2) (gelu), of 1 + exp(-v) (silu): the argument of the
    exponential is rounded a few times, which counts by its size; 2^-19 for Phi's polynomial in 16-bit types."""
    size = v * v / 2 if act == "gelu" else v.abs()
    size = size.clamp_max(150)          # beyond, the exponential is 0
    return 4 * ref.U32 * (4 + size) + (2.0 ** -19 if dtype != F32 and act == "gelu" else 0.0)


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_values(lbp, dtype, act):
    x = numbers(dtype)
    print(f"{act} {dtype} {len(x)}", flush=True)
    y, pre = lbp.linear(x[:, None], torch.ones(1, 1, dtype=dtype, device="cuda"), act=act, want_pre=True)
    assert torch.equal(pre[:, 0], x)
    v = x.double()
    want = v * ndtr(v) if act == "gelu" else v * torch.sigmoid(v)
    e = want.abs() * relative(dtype, act, v)
    # a result below the float32 normal numbers, or one whose exponential is, may be flushed
    flushed = v.abs() * 2.0 ** -126 if act == "gelu" else 2.0 ** -126 * v.abs()
    ref.assert_within(y[:, 0], want, e + flushed + ref.UNIT[dtype] * (want.abs() + e) + ref.TINY[dtype], f"{act} {dtype}")


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_derivatives(lbp, dtype, act):
    s = numbers(dtype)[:, None]
    one = torch.ones(1, 1, dtype=dtype, device="cuda")
    print(f"{act} derivative {dtype} {len(s)}", flush=True)
    got = lbp.linear_backward(torch.ones_like(s), s, one, act=act, saved=s, want_x=False, want_weight=False,
                              want_bias=False, want_residual=True)[3][:, 0]
    v = s[:, 0].double()
    rel = relative(dtype, act, v)
    if act == "gelu":
        phi = torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        want, e = ndtr(v) + v * phi, rel * (ndtr(v) + v.abs() * phi)
    else:
        q, r = torch.sigmoid(v), torch.sigmoid(-v)
        # 1 - q is a difference: its error is a unit of 1
        want, e = q + v * q * r, rel * (q + v.abs() * q * r) + v.abs() * q * (2 * ref.U32 + rel * q)
    e = e + (1 + v.abs()) * 2.0 ** -126
    e = torch.where(torch.isfinite(e), e, torch.zeros_like(e))
    ref.assert_within(got, want, e + ref.UNIT[dtype] * (want.abs() + e) + ref.TINY[dtype], f"{act}' {dtype}")


def test_bound_excludes_a_cancelling_form():
    """The bounds above tell a form that loses the lower tail (1 + erf in float32) from one that does not."""
    for dtype in (F32, BF16, F16):
        v = torch.linspace(-12, -5.2, 200).to(dtype)
        bad = (v.float() * 0.5 * (1 + torch.erf(v.float() * 0.5 ** 0.5))).to(dtype).double()
        w = v.double()
        want = w * ndtr(w)
        e = want.abs() * relative(dtype, "gelu", w)
        over = (bad - want).abs() > e + ref.UNIT[dtype] * (want.abs() + e) + ref.TINY[dtype] + w.abs() * 2.0 ** -126
        assert over.any(), dtype
