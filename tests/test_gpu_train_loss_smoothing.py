"""The mean of the logits in the smoothed loss, against float64 with the rounding of its own
sum as the bound; logits whose mean is far from zero, at row lengths that take every kernel."""
import pytest
import torch

import train_reference as ref
from helpers import ensure_built

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


def make(rows, classes, dtype, level, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.randn(rows, classes, generator=g, device="cuda") * 2 + level + torch.linspace(-3, 1, classes, device="cuda")
    return z.to(dtype), torch.randint(0, classes, (rows,), generator=g, device="cuda")


def expected(z, labels, eps, with_mean=True):
    """(row losses, their bounds) in float64 on the CPU."""
    classes = z.shape[1]
    zz = z.double().cpu()
    zt = zz.gather(1, labels.cpu()[:, None])[:, 0]
    lse, top, mean = torch.logsumexp(zz, 1), zz.amax(1), zz.mean(1)
    want = (1 - eps) * (lse - zt) + eps * (lse - (mean if with_mean else 0.0))
    # float32 sums: a thread adds up to 128 numbers (of rows beyond 256 KB a 1024th of them), 22 more
    # steps join the threads; products and the reciprocal of the count are rounded too
    steps = max(128, classes // 1024 + 1) + 26
    bound = ref.ACT[z.dtype] + steps * ref.U32 * (1 + eps * zz.abs().mean(1)) \
        + 8 * ref.U32 * ((lse - top).abs() + (top - zt).abs() + (top - mean).abs())
    return want, bound


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("classes", [1, 10, 63, 1000, 4100, 12001, 32768, 50001, 65536, 100003, 131073, 262144])
def test_row_losses(lbp, classes, dtype):
    for rows in (3, 70):
        if rows * classes > 8e6:
            continue
        for i, (eps, level) in enumerate(((0.1, 6.0), (1.0, 6.0), (0.5, -9.0))):
            print(f"smoothing {rows} x {classes} {dtype} {eps} {level}", flush=True)
            z, y = make(rows, classes, dtype, level, seed=i)
            want, bound = expected(z, y, eps)
            loss, row, _ = lbp.cross_entropy(z, y, label_smoothing=eps)
            ref.assert_within(row, want, bound, f"smoothing {rows} x {classes} {dtype} {eps} row_loss")
            ref.assert_within(loss, want.mean().reshape(1), (bound.mean() + ref.U32 * want.abs().max()).reshape(1), "loss")
            # a loss without the mean, or with a mean off by a hundredth, would be outside
            mean = z.double().cpu().mean(1)
            assert (((expected(z, y, eps, with_mean=False)[0] - want).abs() > bound) | (mean.abs() < 1)).all()
            assert (eps * 0.01 * mean.abs() > bound)[mean.abs() > 4].all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("classes", [10, 1001, 40004, 131074])
def test_masked_classes(lbp, classes, dtype):
    """Logits of -inf: without smoothing as if they were not there, with it by the formula."""
    eps, scale = 0.25, 8.0
    z, y = make(4, classes, dtype, 1.0, seed=5)
    z[:, ::3] = float("-inf")
    y = torch.full_like(y, 1)
    kept = torch.ones(classes, dtype=torch.bool, device="cuda")
    kept[::3] = False
    print(f"masked {classes} {dtype}", flush=True)
    loss, row, grad = lbp.cross_entropy(z, y, grad_scale=scale)
    assert (grad[:, ~kept] == 0).all() and torch.isfinite(row).all()
    want, bound = expected(z[:, kept], torch.zeros_like(y), 0.0)        # class 1 comes first of those kept
    ref.assert_within(row, want, bound, "row_loss without the masked classes")
    loss, row, grad = lbp.cross_entropy(z, y, label_smoothing=eps, grad_scale=scale)
    assert (row == float("inf")).all() and loss == float("inf")
    p = torch.softmax(z.double(), 1)
    d = p - eps / classes
    d[:, 1] -= 1 - eps
    d *= scale / 4
    e = scale / 4 * (2 * (ref.ACT[dtype] + (max(128, classes // 1024 + 1) + 26) * ref.U32) * p + 4 * ref.U32 * (p + 1 / classes)) \
        + 4 * ref.U32 * d.abs()
    ref.assert_within(grad, d, e + ref.UNIT[dtype] * (d.abs() + e) + ref.TINY[dtype], "smoothed gradient")
