"""The training example with dropout: its gradients against float64, another mask each step, and a
certified network that has none."""
import pytest
import torch

import block_reference as ref
import workloads as wk
from test_gpu_train_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_gradients(example):  # noqa: F811
    """A layer's product sums at most K = 784 terms (128 in the gradients), each sum off by (K + 4) 2^-24 of its
    terms' magnitudes; these are at most sqrt(K) times the sums' own size for terms of random signs, and
    six such sums follow each other: 6 * 788 * 28 * 2^-24 = 2^-7 of the largest value at worst; 2^-9 is asked for."""
    import linear_bound_propagation_amd as lbp
    p = 0.3
    net = example.Net(wk.mlp(example.WIDTHS, 1, 0.01, 1).nodes, dropout=p, seed=7)
    net.steps = 5
    x, labels = example.make_data(128)
    xd, yd = torch.tensor(x, device="cuda"), torch.tensor(labels, device="cuda")
    logits, inputs = net.forward(xd, train=True)
    loss, _, dlogits = lbp.cross_entropy(logits, yd)
    grads = net.backward(dlogits, inputs)
    leaves = [q.double().cpu().requires_grad_() for q in net.parameters()]
    h = torch.tensor(x, dtype=torch.float64)
    scale = 2 ** 32 / (2 ** 32 - round(p * 2 ** 32))
    for i in range(3):
        h = h @ leaves[2 * i].t() + leaves[2 * i + 1]
        if i < 2:
            h = torch.relu(h) * ref.kept(128, 100, p, 7, 5 * 3 + i) * scale
    want = -torch.log_softmax(h, 1)[torch.arange(128), torch.tensor(labels)].mean()
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 2.0 ** -9 * (1 + abs(float(want.detach())))
    for g, leaf in zip(grads, leaves):
        assert float((g.double().cpu() - leaf.grad).abs().max()) <= 2.0 ** -9 * float(leaf.grad.abs().max())


def test_runs_and_certifies(example):  # noqa: F811
    net, losses, before, after = example.run(steps=20, dropout=0.2, log=lambda *a: None)
    assert torch.isfinite(losses).all() and net.steps == 20
    assert all(0 <= certified <= correct <= 64 for correct, certified in (before, after))
    x = torch.tensor(example.make_data(64)[0], device="cuda")
    assert torch.equal(net.forward(x)[0], net.forward(x)[0])            # evaluation drops nothing
    first = net.forward(x, train=True)[0]
    assert torch.equal(first, net.forward(x, train=True)[0])            # a step's mask is its own
    net.steps += 1
    assert not torch.equal(first, net.forward(x, train=True)[0])


def test_without_dropout_nothing_changes(example):  # noqa: F811
    a = example.run(steps=5, log=lambda *a: None)[1]
    b = example.run(steps=5, dropout=0.0, log=lambda *a: None)[1]
    assert torch.equal(a, b)
