"""examples/gated_block.py: the operators as they are used together, against the same block in 64 bits on the CPU."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("gated_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(p, x, r, dy):
    """The block's result and the gradients of sum(y * dy), in 64 bits."""
    leaves = [t.detach().cpu().double().requires_grad_(True) for t in [x, *p]]
    x, norm, shift, w1, b1, w2 = leaves
    h = x + r.cpu().double()
    c = h - h.mean(-1, keepdim=True)
    n = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * norm + shift
    z = n @ w1.t() + b1
    f = w2.shape[1]
    a = z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:]
    y = h + a @ w2.t()
    (y * dy.cpu().double()).sum().backward()
    return y.detach(), [t.grad for t in leaves]


def off(got, want):
    got = got.detach().cpu().double()
    return float((got - want).norm() / want.norm())


def case(example, tokens, width, hidden, **kw):
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    x, r, dy = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3))
    block = example.Block(width, hidden, seed=5, **kw)
    block.shift += 0.1
    block.b1 += 0.05
    y, kept = block.forward(x, r)
    dx, grads = block.backward(dy, kept)
    want, grads64 = reference(block.parameters(), x, r, dy)
    names = ("x", "norm", "shift", "w1", "b1", "w2")
    return off(y, want), [(name, off(got, exact)) for name, got, exact in zip(names, [dx, *grads], grads64)]


def test_block_against_64_bits(gpu, example):
    # a dozen roundings to 8 significant bits stand between inputs and results, each at most 2^-8 relative and independent
    # of the others, a gated product's factors twice over: together under 16 * 2^-8 / sqrt(3)
    bound = 16 * 2.0 ** -8 / math.sqrt(3)
    for tokens, width, hidden in ((1, 64, 200), (37, 130, 262), (300, 512, 1024)):
        print("[case] gated block", tokens, width, hidden, flush=True)
        y, grads = case(example, tokens, width, hidden)
        assert y < bound, y
        for name, d in grads:
            assert d < bound, (name, d)


def test_block_with_8_bit_products(gpu, example):
    # one product each of y, da and dw2 has both operands rounded to E4M3, each within 2^-4 of its value: 2 * 2^-4 of the
    # product, on top of the 16-bit block's bound; what da reaches carries it on
    bound = 16 * 2.0 ** -8 / math.sqrt(3) + 2 * 2.0 ** -4 + 2.0 ** -8
    for tokens, width, hidden in ((1, 64, 208), (37, 144, 272), (300, 512, 1024)):
        print("[case] gated block in 8 bits", tokens, width, hidden, flush=True)
        y, grads = case(example, tokens, width, hidden, eight_bits=True)
        assert y < bound, y
        for name, d in grads:
            assert d < bound, (name, d)


def test_serving_in_8_bits(gpu, example):
    # two products in a row with both operands within 2^-4 of their values, the first one's result a product of two factors
    # that both carry its error (each no steeper than 1.1): (2 * 2.2 + 2) * 2^-4, next to what the residual carries unrounded
    for tokens, width, hidden in ((1, 256, 512), (64, 512, 1024), (333, 1024, 2048)):
        g = torch.Generator(device="cuda")
        g.manual_seed(tokens)
        x, r = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(2))
        block = example.Block(width, hidden, seed=6)
        y, _ = block.forward(x, r)
        got = example.Serving(block).forward(x, r)
        assert got.shape == y.shape and got.dtype == y.dtype
        assert off(got, y.cpu().double()) < 6.4 * 2.0 ** -4, (tokens, off(got, y.cpu().double()))


def test_a_step_as_a_graph(gpu, example):
    """Forward and backward captured together and replayed with other inputs, eager work in between."""
    for eight in (False, True):
        block = example.Block(256, 512, eight_bits=eight, seed=7)
        sets = []
        for seed in (1, 2):
            g = torch.Generator(device="cuda")
            g.manual_seed(seed)
            sets.append([torch.randn(200, 256, generator=g, device="cuda").bfloat16() for _ in range(3)])

        def step(x, r, dy):
            y, kept = block.forward(x, r)
            dx, grads = block.backward(dy, kept)
            return [y, dx, *grads]
        want = [step(*s) for s in sets]
        fed = [t.clone() for t in sets[0]]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(*fed)
        for i in (0, 1, 0, 1):
            for t, v in zip(fed, sets[i]):
                t.copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i])), (eight, i)
            assert all(torch.equal(a, b) for a, b in zip(step(*sets[1 - i]), want[1 - i]))
