"""Trains the 784-100-100-10 ReLU network on synthetic classes with the package's training
operators (fused linear layers and their gradients, cross entropy, gradient clipping), then
certifies the trained network with CROWN: how many inputs keep their class under every
perturbation of at most eps.

    python examples/train_and_certify.py [--steps 200] [--eps 0.01]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_bound_propagation_amd as lbp  # noqa: E402
import workloads as wk  # noqa: E402

WIDTHS = (784, 100, 100, 10)


def make_data(n: int, seed: int = 0):
    """n inputs in [0, 1]^784 of ten classes: a random pattern per class, noise around it."""
    rng = np.random.default_rng([seed, 0])
    patterns = rng.random((WIDTHS[-1], WIDTHS[0]))
    rng = np.random.default_rng([seed, 1])
    labels = rng.integers(0, WIDTHS[-1], n)
    x = np.clip(patterns[labels] + 0.5 * rng.standard_normal((n, WIDTHS[0])), 0, 1)
    return x.astype(np.float32), labels.astype(np.int64)


class Net:
    """The network's parameters on the device: [(weight, bias)] per layer."""

    def __init__(self, nodes, device="cuda"):
        self.layers = [(torch.tensor(n.weight, device=device), torch.tensor(n.bias, device=device))
                       for n in nodes if n.op == "linear"]

    def forward(self, x):
        """Logits, and the input of every layer (a ReLU's output is what its gradient needs)."""
        inputs = [x]
        for i, (w, b) in enumerate(self.layers):
            last = i + 1 == len(self.layers)
            inputs.append(lbp.linear(inputs[-1], w, b, act="none" if last else "relu"))
        return inputs[-1], inputs[:-1]

    def backward(self, dlogits, inputs):
        """Gradients in the order of `parameters`."""
        grads, d = [], dlogits
        for i in reversed(range(len(self.layers))):
            last = i + 1 == len(self.layers)
            saved = None if last else inputs[i + 1]
            d, dw, db, _ = lbp.linear_backward(d, inputs[i], self.layers[i][0], act="none" if last else "relu",
                                               saved=saved, want_x=i > 0)
            grads = [dw, db] + grads
        return grads

    def parameters(self):
        return [p for layer in self.layers for p in layer]

    def step(self, x, labels, lr: float, max_norm: float):
        """One step of gradient descent; returns (loss, gradient norm), both on the device."""
        logits, inputs = self.forward(x)
        loss, _, dlogits = lbp.cross_entropy(logits, labels, dlogits=logits)    # the gradient over the logits
        grads = self.backward(dlogits, inputs)
        norm, grads = lbp.clip_grad_norm(grads, max_norm)
        for p, g in zip(self.parameters(), grads):
            p.add_(g, alpha=-lr)
        return loss, norm


def certify(net: Net, nodes, x: np.ndarray, labels: np.ndarray, eps: float):
    """(correct, certified): inputs classified as their label, and those whose label holds for
    the whole ball of radius eps (CROWN bounds of all nine margins positive)."""
    it = iter(net.layers)
    for n in nodes:
        if n.op == "linear":
            w, b = next(it)
            n.weight, n.bias = w.cpu().numpy(), b.cpu().numpy()
    device = lbp.DeviceNet(nodes)
    xd = torch.tensor(x, device="cuda")
    eye = np.eye(WIDTHS[-1], dtype=np.float32)
    C = np.stack([np.delete(eye[t] - eye, t, 0) for t in labels])
    out = lbp.crown(device, xd, eps, torch.tensor(C, device="cuda"), "crown")
    _, count = lbp.verify(out["lb"])
    logits, _ = net.forward(xd)
    correct = (logits.argmax(1).cpu().numpy() == labels).sum()
    return int(correct), int(count)


def run(steps: int = 200, batch: int = 128, eps: float = 0.01, lr: float = 0.1, max_norm: float = 1.0, n_test: int = 64,
        log=print):
    nodes = wk.mlp(WIDTHS, 1, eps, 1).nodes
    net = Net(nodes)
    x, labels = make_data(batch * 16 + n_test)
    test = slice(batch * 16, None)
    xd, yd = torch.tensor(x, device="cuda"), torch.tensor(labels, device="cuda")
    before = certify(net, nodes, x[test], labels[test], eps)
    log(f"before training: {before[0]} of {n_test} correct, {before[1]} certified at eps {eps}")
    losses = []
    for t in range(steps):
        part = slice(t % 16 * batch, (t % 16 + 1) * batch)
        loss, norm = net.step(xd[part], yd[part], lr, max_norm)
        losses.append(loss)
        if t % 50 == 0 or t + 1 == steps:
            log(f"step {t}: loss {float(loss):.4f}, gradient norm {float(norm):.3f}")
    after = certify(net, nodes, x[test], labels[test], eps)
    log(f"after training: {after[0]} of {n_test} correct, {after[1]} certified at eps {eps}")
    return net, torch.cat(losses), before, after


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--eps", type=float, default=0.01)
    a = ap.parse_args()
    run(steps=a.steps, eps=a.eps)
