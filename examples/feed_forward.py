"""A transformer's feed-forward block on the linear-layer operators: training steps, then decoding.

    Y = act(X W1^T + b1) W2^T + b2 + X

Forward: linear (bias, activation, the pre-activation kept), linear (bias, the residual added).
Backward, from dY = dL/dY:
    dW2 += dY^T H          linear_wgrad, added to the fp32 gradient
    db2 += sum dY          act_grad, sums only
    dZ   = (dY W2) act'(Z) linear_dgrad, with db1 += its column sums
    dW1 += dZ^T X          linear_wgrad
    dX   = dZ W1 + dY      linear_dgrad, then the residual's path
H is act(Z), recomputed by nobody: the forward pass keeps it as the second product's input.

The block is fitted to a fixed random target, in bf16 with fp32 master weights; every micro-batch adds to the same
fp32 gradients.  Then single tokens go through it, as a decoding loop would send them, and must agree with the batch.

    python examples/feed_forward.py [--tokens 2048] [--width 1024] [--hidden 4096] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dense_tiled_gemm_04_gb300 import Gemm  # noqa: E402


class FeedForward:
    def __init__(self, width: int, hidden: int, act: str = "gelu_tanh", device=0, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5

        self.gemm, self.act = Gemm(device), act
        self.master = {"W1": weight(hidden, width), "b1": torch.zeros(hidden, device="cuda"),
                       "W2": weight(width, hidden), "b2": torch.zeros(width, device="cuda")}
        self.grad = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.moments = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in self.master.items()}
        self.steps = 0
        self.cast()

    def cast(self):
        """The weights that the products read: bf16 (biases stay fp32)."""
        self.W1, self.W2 = self.master["W1"].bfloat16(), self.master["W2"].bfloat16()

    def forward(self, X, keep=True):
        """Y, and what the backward pass needs."""
        Z = torch.empty((X.shape[0], self.W1.shape[0]), dtype=X.dtype, device=X.device) if keep else None
        H = self.gemm.linear(X, self.W1, self.master["b1"], act=self.act, preact=Z)
        Y = self.gemm.linear(H, self.W2, self.master["b2"], residual=X)
        return Y, (X, Z, H)

    def backward(self, dY, saved):
        """Adds to the gradients; returns dL/dX."""
        X, Z, H = saved
        g = self.grad
        self.gemm.linear_wgrad(dY, H, out=g["W2"], beta=1.0)
        self.gemm.act_grad(dY, dbias=g["b2"], beta_bias=1.0, sums_only=True)
        dZ = self.gemm.linear_dgrad(dY, self.W2, Z, act=self.act, dbias=g["b1"], beta_bias=1.0)
        self.gemm.linear_wgrad(dZ, X, out=g["W1"], beta=1.0)
        return self.gemm.linear_dgrad(dZ, self.W1).add_(dY)

    def step(self, rate: float, beta1: float = 0.9, beta2: float = 0.99):
        """An Adam step on the master weights; clears the gradients."""
        self.steps += 1
        for k, w in self.master.items():
            g, (m, v) = self.grad[k], self.moments[k]
            m.lerp_(g, 1 - beta1)
            v.lerp_(g * g, 1 - beta2)
            w.sub_(rate / (1 - beta1 ** self.steps) * m / ((v / (1 - beta2 ** self.steps)).sqrt() + 1e-8))
            g.zero_()
        self.cast()


def train(tokens=2048, width=1024, hidden=4096, steps=20, micro_batches=2, rate=None, seed=0):
    """(losses, the largest difference of a token decoded alone from its row of the batch)."""
    block = FeedForward(width, hidden, seed=seed)
    rate = rate or 1.0 / hidden  # a step moves each of an output's `hidden` terms
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    X = torch.randn((tokens, width), generator=gen, device="cuda").bfloat16()
    target = torch.randn((tokens, width), generator=gen, device="cuda").bfloat16()
    losses = []
    for _ in range(steps):
        loss = 0.0
        for x, t in zip(X.chunk(micro_batches), target.chunk(micro_batches)):
            Y, saved = block.forward(x)
            diff = Y.float() - t.float()
            loss += diff.square().sum()
            block.backward((diff * (2.0 / tokens)).bfloat16(), saved)
        block.step(rate)
        losses.append(loss.item() / (tokens * width))
    batch, _ = block.forward(X[:8], keep=False)
    alone = torch.cat([block.forward(X[i:i + 1], keep=False)[0] for i in range(8)])
    if block.gemm.sync_status() != 0:
        raise RuntimeError("a kernel reported a failure")
    return losses, (batch.float() - alone.float()).abs().max().item()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("width", 1024), ("hidden", 4096), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    losses, off = train(a.tokens, a.width, a.hidden, a.steps)
    print("loss " + " ".join(f"{x:.4f}" for x in losses))
    print(f"a token alone and in its batch differ by at most {off:.4g}")


if __name__ == "__main__":
    main()
