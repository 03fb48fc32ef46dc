"""examples/feed_forward.py: the operators as they are used together, against the same block in 64 bits on the CPU."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")


@pytest.fixture(scope="module")
def ff():
    spec = importlib.util.spec_from_file_location("feed_forward", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(p, x, r, dy):
    """The block's result and the gradients of sum(y * dy), in 64 bits."""
    leaves = [t.detach().cpu().double().requires_grad_(True) for t in [x, *p]]
    x, norm, w1, b1, w2 = leaves
    h = x + r.cpu().double()
    n = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * norm
    z = n @ w1.t() + b1
    a = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    y = h + a @ w2.t()
    (y * dy.cpu().double()).sum().backward()
    return y.detach(), [t.grad for t in leaves]


def off(got, want):
    got = got.detach().cpu().double()
    return float((got - want).norm() / want.norm())


def test_block_against_64_bits(gpu, ff):
    # a dozen roundings to 8 significant bits stand between inputs and results, each at most 2^-8 relative and
    # independent of the others: together under 12 * 2^-8 / sqrt(3), taken without the averaging over a norm's terms
    bound = 12 * 2.0 ** -8 / math.sqrt(3)
    for tokens, width, hidden in ((1, 64, 200), (37, 130, 264), (300, 512, 1024)):
        print("[case] feed forward", tokens, width, hidden, flush=True)
        g = torch.Generator(device="cuda")
        g.manual_seed(tokens)
        x, r, dy = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3))
        block = ff.Block(width, hidden, seed=5)
        y, kept = block.forward(x, r)
        dx, grads = block.backward(dy, kept)
        want, grads64 = reference(block.parameters(), x, r, dy)
        assert off(y, want) < bound
        for name, got, exact in zip(("x", "norm", "w1", "b1", "w2"), [dx, *grads], grads64):
            assert off(got, exact) < bound, (name, off(got, exact))


def test_serving_in_8_bits(gpu, ff):
    # each product's inputs and weights are rounded to 8 bits: E4M3 within 2^-4 relative of each value, int8 within
    # amax / 254 of a row whose normal entries have amax below 5 standard deviations; the two products' errors add to
    # what the residual carries unrounded
    for tokens, width, hidden in ((1, 256, 512), (64, 512, 1024), (333, 1024, 2048)):
        g = torch.Generator(device="cuda")
        g.manual_seed(tokens)
        x, r = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(2))
        block = ff.Block(width, hidden, seed=6)
        y, _ = block.forward(x, r)
        for dtype, bound in ((torch.float8_e4m3fn, 4 * 2.0 ** -4), (torch.int8, 4 * 5 / 254)):
            got = ff.Serving(block, dtype).forward(x, r)
            assert got.shape == y.shape and got.dtype == y.dtype
            assert off(got, y.cpu().double()) < bound, (tokens, dtype, off(got, y.cpu().double()))


def test_training_lowers_the_loss(gpu, ff):
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x, r = (torch.randn(512, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    target, _ = ff.Block(256, 512, seed=2).forward(x, r)
    losses = ff.train(ff.Block(256, 512, seed=3), x, r, target, steps=8, rate=0.05)
    assert all(math.isfinite(v) for v in losses) and losses[-1] < 0.9 * losses[0], losses
