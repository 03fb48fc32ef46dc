"""Matrices of more than 2^31 elements: the layer norm, its backward pass, the blocks and the gated backward pass.

Rows at the start, past 2^31 bytes and elements, and at the end are the bits that the same rows give on their own (every row,
and every block, stands by itself, and a slice of 1200 rows runs the same kernels); products and sums over rows are compared
with 64 bits.
"""
import pytest
import torch

from test_layers_gpu import say, u

ROWS, D = 530_000, 4100  # 2.2e9 elements; 4100 ends inside a chunk of 8 and inside a block of 128


def slices():
    return [slice(at, at + 1200) for at in (0, 261_000, ROWS // 128 * 128 - 12_800, ROWS - 1200)]


def big(seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(ROWS, D, dtype=dtype, device="cuda")
    for part in x.split(40_000):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return x


def same(a, b, what):
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), what


@pytest.mark.gpu
def test_layer_norm_and_its_backward_pass(gpu):
    say("layer norm", ROWS, D)
    x, r = big(1), big(2)
    w, b = 1 + 0.1 * torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    got = gpu.add_layer_norm(x, w, b, residual=r, save_stats=True)
    for s in slices():
        one = gpu.add_layer_norm(x[s], w, b, residual=r[s], save_stats=True)
        for t, want, what in zip(got, one, got._fields):
            if what != "scale":
                same(t[s], want, (what, s))
    parts = [r[s].clone() for s in slices()]
    codes = gpu.add_layer_norm(x, w, b, residual=r, out_dtype=torch.float8_e4m3fn, h_out=r)
    for s, kept in zip(slices(), parts):
        same(codes.h[s], got.h[s], s)
        one = gpu.add_layer_norm(x[s], w, b, residual=kept, out_dtype=torch.float8_e4m3fn)
        same(codes.y[s], one.y, ("codes", s))
        same(codes.scale[s], one.scale, ("scale", s))
    h, dy = got.h, x
    del codes, r
    back = gpu.add_layer_norm_backward(dy, h, w, got.mean, got.rstd, dh=dy)
    for s in slices():
        one = gpu.add_layer_norm_backward(dy[s], h[s], w, got.mean[s], got.rstd[s], dh=dy[s])
        same(back.dx[s], one.dx, ("dx", s))
    # sums over rows, in fp64: within (rows + 8) u of the sum of magnitudes
    dw, db, size_w, size_b = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(4))
    for at in range(0, ROWS, 20_000):
        s = slice(at, min(ROWS, at + 20_000))
        t = dy[s].double()
        xhat = (h[s].double() - got.mean[s].double()[:, None]) * got.rstd[s].double()[:, None]
        db += t.sum(0)
        size_b += t.abs().sum(0)
        dw += (t * xhat).sum(0)
        size_w += (t * xhat).abs().sum(0)
    assert bool(((back.dweight.double() - dw).abs() <= (ROWS + 8) * u * size_w).all())
    assert bool(((back.dbias.double() - db).abs() <= (ROWS + 8) * u * size_b).all())


@pytest.mark.gpu
@pytest.mark.parametrize("high", [1, 128])
def test_blocks(gpu, high):
    say("quantize blocks", ROWS, D, high)
    x = big(3)
    got = gpu.quantize_blocks(x, block=(high, 128))
    for at in (0, 261_120, ROWS // 128 * 128 - 12_800):  # whole blocks of rows
        s = slice(at, at + 1280)
        one = gpu.quantize_blocks(x[s], block=(high, 128))
        same(got.q[s], one.q, s)
        same(got.scale[at // high:(at + 1280) // high], one.scale, s)
    del got
    got = gpu.quantize_blocks(x, block=(high, 128), transpose=True)
    assert got.q.shape == (D, (ROWS + 15) // 16 * 16)
    for at in (0, 261_120, ROWS // 128 * 128 - 12_800):
        one = gpu.quantize_blocks(x[at:at + 1280], block=(high, 128), transpose=True)
        same(got.q[:, at:at + 1280], one.q, at)
        same(got.scale[:, at // 128:at // 128 + 10], one.scale, at)
    last = ROWS // 128 * 128
    one = gpu.quantize_blocks(x[last:], block=(high, 128), transpose=True)
    same(got.q[:, last:], one.q, "the last rows")


@pytest.mark.gpu
def test_gated_backward(gpu):
    """Pre-activations and dz of more than 2^31 elements; tolerances as in test_gated.py, of the plain gate and of relu."""
    M, N, K = ROWS, D // 2, 64
    say("gated backward", M, N, K)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = (torch.randn(n, K, generator=g, device="cuda").bfloat16() for n in (M, 2 * N))
    z, dy = big(6), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    for part in dy.split(80_000):
        part.copy_(0.1 * torch.randn(part.shape, generator=g, device="cuda"))
    for act in ("none", "relu"):
        got = gpu.gated_linear_backward(dy, x, w, z, activation=act)

        def dz64(s):
            gate, up, d = z[s, :N].double(), z[s, N:].double(), dy[s].double()
            value, slope = (gate, torch.ones_like(gate)) if act == "none" else (gate.clamp_min(0), (gate > 0).double())
            return torch.cat((d * up * slope, d * value), 1)
        w64 = w.double()
        for s in slices():
            dz = dz64(s)
            size = torch.mm(dz.abs(), w64.abs())
            want = torch.mm(dz, w64)
            # dz in bf16, three roundings before it, the sums, and the result in bf16
            tol = (2.0 ** -8 + (2 * N + 8) * u) * size + 2.0 ** -8 * want.abs() + 2.0 ** -126
            assert bool(((got.dx[s].double() - want).abs() <= tol).all()), (act, s)
        dw, size_w = (torch.zeros(2 * N, K, dtype=torch.float64, device="cuda") for _ in range(2))
        db, size_b = (torch.zeros(2 * N, dtype=torch.float64, device="cuda") for _ in range(2))
        for at in range(0, M, 20_000):
            s = slice(at, min(M, at + 20_000))
            dz, xs = dz64(s).t().contiguous(), x[s].double()
            dw += torch.mm(dz, xs)
            size_w += torch.mm(dz.abs(), xs.abs())
            db += dz.sum(1)
            size_b += dz.abs().sum(1)
        assert bool(((got.dweight.double() - dw).abs() <= (2.0 ** -8 + (M + 8) * u) * size_w + 2.0 ** -8 * dw.abs()).all()), act
        assert bool(((got.dbias.double() - db).abs() <= (M + 8) * u * size_b + 2.0 ** -8 * db.abs()).all()), act
