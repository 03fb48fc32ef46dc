"""A pre-norm block with a gated feed-forward part on this package's operators, in 16 bits and with 8-bit products.

    python examples/gated_block.py [--tokens 4096] [--width 4096] [--hidden 8192] [--steps 10]

One block is h = x + residual; n = layer_norm(h); a = act(Wg n + bg) * (Wu n + bu); y = h + Wd a.  `Block.forward` and
`Block.backward` are a training step's two passes.  With ``eight_bits`` the down projection's three products (its result and
both gradients) run on E4M3 codes with one scale per block of 128 along each product's own sum; everything else stays in 16
bits.  `Serving` keeps 8-bit weights and runs the block for prompts and for single tokens: the norm leaves 8-bit rows with
scales for the gated projection, whose result is quantised in blocks for the down projection.  Prints the loss of a few
steps of gradient descent, how far 8 bits are from 16, and times.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import dense_tiled_gemm_amd as gb  # noqa: E402
from feed_forward import clock, train  # noqa: E402


class Block:
    def __init__(self, width, hidden, dtype=torch.bfloat16, activation="silu", eight_bits=False, seed=0):
        if eight_bits and (width % 16 or hidden % 16):
            raise ValueError("8-bit products need a width and a hidden size that are multiples of 16")
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        new = lambda *shape, std: (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
        self.activation, self.eight_bits = activation, eight_bits
        self.norm, self.shift = torch.ones(width, dtype=dtype, device="cuda"), torch.zeros(width, dtype=dtype, device="cuda")
        self.w1, self.b1 = new(2 * hidden, width, std=width ** -0.5), torch.zeros(2 * hidden, dtype=dtype, device="cuda")
        self.w2 = new(width, hidden, std=hidden ** -0.5)

    def parameters(self):
        return [self.norm, self.shift, self.w1, self.b1, self.w2]

    def forward(self, x, residual):
        """(y, what the backward pass needs)."""
        n = gb.add_layer_norm(x, self.norm, self.shift, residual=residual, save_stats=True)
        a, z = gb.gated_linear(n.y, self.w1, bias=self.b1, activation=self.activation, save_preact=True)
        if self.eight_bits:
            q, w = gb.quantize_blocks(a), gb.quantize_blocks(self.w2, block=(128, 128))
            y = gb.block_linear(q.q, w.q, q.scale, w.scale, residual=n.h, out_dtype=x.dtype)
        else:
            y = gb.linear(a, self.w2, residual=n.h)
        return y, (n, a, z)

    def down_backward(self, dy, a):
        """Gradients of a and w2: sums over the width and over the tokens."""
        if not self.eight_bits:
            g = gb.linear_backward(dy, a, self.w2, bias_grad=False)
            return g.dx, g.dweight
        q, w = gb.quantize_blocks(dy), gb.quantize_blocks(self.w2, block=(128, 128), transpose=True)
        da = gb.block_linear(q.q, w.q, q.scale, w.scale, out_dtype=dy.dtype)
        q, p = gb.quantize_blocks(dy, transpose=True), gb.quantize_blocks(a, transpose=True)
        return da, gb.block_linear(q.q, p.q, q.scale, p.scale, out_dtype=dy.dtype)

    def backward(self, dy, kept):
        """(gradient of x and of residual alike, gradients of the parameters)."""
        n, a, z = kept
        da, dw2 = self.down_backward(dy, a)
        first = gb.gated_linear_backward(da, n.y, self.w1, z, activation=self.activation)
        norm = gb.add_layer_norm_backward(first.dx, n.h, self.norm, n.mean, n.rstd, dh=dy)  # dy also reaches h past the products
        return norm.dx, [norm.dweight, norm.dbias, first.dweight, first.dbias, dw2]


class Serving:
    def __init__(self, block):
        self.block = block
        self.q1, self.s1 = gb.quantize_rows(block.w1)
        self.q2, self.s2 = gb.quantize_blocks(block.w2, block=(128, 128))

    def forward(self, x, residual):
        b = self.block
        n = gb.add_layer_norm(x, b.norm, b.shift, residual=residual, out_dtype=torch.float8_e4m3fn)
        a = gb.gated_linear(n.y, self.q1, bias=b.b1, activation=b.activation, x_scale=n.scale, weight_scale=self.s1, out_dtype=x.dtype)
        q = gb.quantize_blocks(a)
        return gb.block_linear(q.q, self.q2, q.scale, self.s2, residual=n.h, out_dtype=x.dtype)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    if not torch.cuda.is_available():
        raise SystemExit("gated_block.py needs a GPU")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, residual = (torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16() for _ in range(2))
    target, _ = Block(a.width, a.hidden, seed=2).forward(x, residual)
    for eight in (False, True):
        block = Block(a.width, a.hidden, eight_bits=eight, seed=3)
        losses = train(block, x, residual, target, a.steps, rate=0.05)
        y, kept = block.forward(x, residual)
        print("%s: loss %s; forward %.0f us, backward %.0f us"
              % ("8-bit down projection" if eight else "16 bits", " ".join("%.4f" % v for v in losses),
                 clock(lambda: block.forward(x, residual)), clock(lambda: block.backward(y, kept))))
    serving = Serving(block)
    off = (serving.forward(x, residual).float() - y.float()).norm() / y.float().norm()
    one, one_r = x[:1], residual[:1]
    print("serving in 8 bits: %.2f %% from the trained block, prompt of %d tokens %.0f us, one token %.0f us (16 bits %.0f us)"
          % (100 * float(off), a.tokens, clock(lambda: serving.forward(x, residual)), clock(lambda: serving.forward(one, one_r)),
             clock(lambda: block.forward(one, one_r))))


if __name__ == "__main__":
    main()
