"""A pre-norm feed-forward block on this package's operators: trained in 16 bits, then served in 8.

    python examples/feed_forward.py [--tokens 4096] [--width 4096] [--hidden 8192] [--steps 10]

One block is h = x + residual; y = h + W2 act(W1 norm(h) + b1).  `Block.forward` and `Block.backward` are a training
step's two passes (the norm with the residual's addition, two products with their epilogues, and their gradients);
`Serving` holds the weights in E4M3 or int8 with one scale per row and runs the same block for prompts and for single
tokens: the norm leaves 8-bit rows with scales, the first product its activations in 16 bits, which are quantised again
for the second.  Prints the loss of a few steps of gradient descent, how far 8 bits are from 16, and times.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_tiled_gemm_amd as gb  # noqa: E402


class Block:
    def __init__(self, width, hidden, dtype=torch.bfloat16, activation="gelu_tanh", seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        new = lambda *shape, std: (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
        self.activation = activation
        self.norm = torch.ones(width, dtype=dtype, device="cuda")
        self.w1, self.b1 = new(hidden, width, std=width ** -0.5), torch.zeros(hidden, dtype=dtype, device="cuda")
        self.w2 = new(width, hidden, std=hidden ** -0.5)

    def parameters(self):
        return [self.norm, self.w1, self.b1, self.w2]

    def forward(self, x, residual):
        """(y, what the backward pass needs)."""
        n = gb.add_rms_norm(x, self.norm, residual=residual, save_rstd=True)
        a, z = gb.linear(n.y, self.w1, bias=self.b1, activation=self.activation, save_preact=True)
        return gb.linear(a, self.w2, residual=n.h), (n, a, z)

    def backward(self, dy, kept):
        """(gradient of x and of residual alike, gradients of the parameters)."""
        n, a, z = kept
        second = gb.linear_backward(dy, a, self.w2, bias_grad=False)
        first = gb.linear_backward(second.dx, n.y, self.w1, preact=z, activation=self.activation)
        dx, dnorm = gb.add_rms_norm_backward(first.dx, n.h, self.norm, n.rstd, dh=dy)  # dy also reaches h past the products
        return dx, [dnorm, first.dweight, first.dbias, second.dweight]


class Serving:
    def __init__(self, block, dtype=torch.float8_e4m3fn):
        self.block, self.dtype = block, dtype
        self.q1, self.s1 = gb.quantize_rows(block.w1, dtype)
        self.q2, self.s2 = gb.quantize_rows(block.w2, dtype)

    def forward(self, x, residual):
        b = self.block
        n = gb.add_rms_norm(x, b.norm, residual=residual, out_dtype=self.dtype)
        a = gb.linear(n.y, self.q1, bias=b.b1, activation=b.activation, x_scale=n.scale, weight_scale=self.s1, out_dtype=x.dtype)
        q = gb.quantize_rows(a, self.dtype)
        return gb.linear(q.q, self.q2, residual=n.h, x_scale=q.scale, weight_scale=self.s2, out_dtype=x.dtype)


def train(block, x, residual, target, steps, rate):
    """A few steps of gradient descent on the mean squared distance from `target`, each of `rate` times a parameter's own
    length; the losses."""
    losses = []
    for _ in range(steps):
        y, kept = block.forward(x, residual)
        off = y.float() - target.float()
        losses.append(float(off.square().mean()))
        _, grads = block.backward((off * (2.0 / off.shape[0])).to(y.dtype), kept)
        for p, g in zip(block.parameters(), grads):
            p -= (rate * p.float().norm().clamp_min(1.0) / g.float().norm().clamp_min(1e-12)) * g
    return losses


def clock(call, times=20):
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(times):
        call()
    torch.cuda.synchronize()
    return (time.perf_counter() - start) / times * 1e6


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    if not torch.cuda.is_available():
        raise SystemExit("feed_forward.py needs a GPU")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, residual = (torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16() for _ in range(2))
    teacher, block = Block(a.width, a.hidden, seed=2), Block(a.width, a.hidden, seed=3)
    target, _ = teacher.forward(x, residual)
    losses = train(block, x, residual, target, a.steps, rate=0.05)
    print("loss: " + " ".join("%.4f" % v for v in losses))
    y, kept = block.forward(x, residual)
    print("training: forward %.0f us, backward %.0f us" % (clock(lambda: block.forward(x, residual)), clock(lambda: block.backward(y, kept))))
    for dtype in (torch.float8_e4m3fn, torch.int8):
        serving = Serving(block, dtype)
        off = (serving.forward(x, residual).float() - y.float()).norm() / y.float().norm()
        one, one_r = x[:1], residual[:1]
        print("%s: %.2f %% from 16 bits, prompt of %d tokens %.0f us, one token %.0f us (16 bits %.0f us)"
              % (str(dtype)[6:], 100 * float(off), a.tokens, clock(lambda: serving.forward(x, residual)),
                 clock(lambda: serving.forward(one, one_r)), clock(lambda: block.forward(one, one_r))))


if __name__ == "__main__":
    main()
