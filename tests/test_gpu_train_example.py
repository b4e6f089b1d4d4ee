"""The training example end to end: its losses follow the same training in float64, and the
trained network is certified where the untrained one is not."""
import os
import sys

import numpy as np
import pytest
import torch

from helpers import ROOT, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    ensure_built()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_and_certify as m
    return m


def float64_losses(example, steps, batch, lr, max_norm):
    """The same training by autograd in float64 on the CPU."""
    import workloads as wk
    nodes = wk.mlp(example.WIDTHS, 1, 0.01, 1).nodes
    params = [torch.tensor(p, dtype=torch.float64, requires_grad=True)
              for n in nodes if n.op == "linear" for p in (n.weight, n.bias)]
    x, labels = example.make_data(batch * 16 + 64)
    out = []
    for t in range(steps):
        h = torch.tensor(x[t % 16 * batch:(t % 16 + 1) * batch], dtype=torch.float64)
        y = torch.tensor(labels[t % 16 * batch:(t % 16 + 1) * batch])
        for i in range(0, len(params), 2):
            h = h @ params[i].t() + params[i + 1]
            if i + 2 < len(params):
                h = torch.relu(h)
        loss = -torch.log_softmax(h, 1)[torch.arange(batch), y].mean()
        grads = torch.autograd.grad(loss, params)
        norm = torch.sqrt(sum((g * g).sum() for g in grads))
        s = min(1.0, max_norm / float(norm))
        with torch.no_grad():
            for p, g in zip(params, grads):
                p -= lr * s * g
        out.append(float(loss.detach()))
    return np.array(out)


def test_training_follows_float64_and_certifies(example):
    steps, batch, lr, max_norm = 120, 128, 0.1, 1.0
    net, losses, before, after = example.run(steps=steps, batch=batch, lr=lr, max_norm=max_norm)
    want = float64_losses(example, steps, batch, lr, max_norm)
    got = losses.double().cpu().numpy()
    # float32 rounding grows along the trajectory; a wrong gradient moves the loss by far more
    assert np.all(np.abs(got - want) <= 1e-3 * (1 + np.abs(want))), np.abs(got - want).max()
    assert want[-1] < 0.1 * want[0]
    assert after[0] >= 60 and after[1] >= 48 and before[1] <= 8, (before, after)
