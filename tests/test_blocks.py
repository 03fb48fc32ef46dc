"""8-bit matrices with one scale per block of 128, and their product, against plain implementations in 64 bits.

Where the tolerances come from (u = 2^-24).  A scale is one division; codes are taken from v times 448 / amax, two roundings
before that of E4M3.  A product's sums of 8-bit floats are known to within eight_bit_tol of the scaled operands (a block's
scales are one factor of its sums), sums for fp32 results, whose operands are widened, to within sum_tol: its K u has one
rounding per term, the K / 128 + 4 for the blocks' sums and the scales come on top.  Bias, activation and residual as for
the other products.
"""
import ctypes
import itertools

import pytest
import torch

import dense_tiled_gemm_amd as gb
from test_gated import eight_bit_tol, sum_tol
from test_layers_gpu import ACTS, DT, act64, close, gen, guarded, options, randn, say, u

BAD, UNSUP = gb.ERR_INVALID_VALUE, gb.ERR_UNSUPPORTED
F8 = torch.float8_e4m3fn


def up(n, m):
    return -(-n // m)


def spread(scale, rows, cols, high):
    """A block's scale at each of its entries."""
    s = scale.cpu().double()
    return (s.repeat_interleave(128, 0)[:rows] if high > 1 else s).repeat_interleave(128, 1)[:, :cols]


def block_max(v, high):
    rows, cols = v.shape
    t = torch.nn.functional.pad(v.abs(), (0, -cols % 128, 0, -rows % high))
    return t.unflatten(0, (-1, high)).unflatten(2, (-1, 128)).amax((1, 3))


def check_codes(q, scale, v, high, what):
    """q and scale against the exact values v (rows, cols)."""
    rows, cols = v.shape
    v = v.double()
    want = torch.clamp(block_max(v, high) / 448, min=2.0 ** -100)
    assert scale.shape == want.shape and scale.dtype == torch.float32, (what, scale.shape, want.shape)
    s = scale.cpu().double()
    assert bool(((s - want).abs() <= 2 * u * want).all()), what
    full = spread(want, rows, cols, high)
    got, r = q.float().double().cpu()[:, :cols], v / full
    assert not bool(q.float()[:, cols:].any()), what
    near = r.abs() * (1 + 8 * u)  # a value that the roundings may carry past a power of two is rounded as there
    half = torch.exp2(torch.floor(torch.log2(near.clamp_min(2.0 ** -6))) - 4)
    assert bool(((got - r).abs() <= half + 8 * u * r.abs()).all()), what
    top = block_max(got, high)
    assert bool((top[want > 2.0 ** -99] == 448).all()), what


SIZES = [(1, 1), (1, 16), (1, 8192), (3, 127), (5, 128), (17, 129), (16, 4096), (128, 128), (127, 300), (129, 1000), (130, 2056), (300, 77),
         (1000, 2000), (513, 1031), (2049, 512)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", SIZES)
def test_quantize_blocks(gpu, rows, d):
    for dt, high, transpose in itertools.product(DT, (1, 128), (False, True)):
        seed = rows + d + high
        x = (randn(seed, rows, d, std=3.0) * torch.exp(randn(seed + 1, rows, 1))).to(DT[dt])
        say("quantize blocks", rows, d, dt, high, transpose, "seed", seed)
        got = gpu.quantize_blocks(x.cuda(), block=(high, 128), transpose=transpose)
        v = x.t() if transpose else x
        assert got.q.shape == ((d, up(rows, 16) * 16) if transpose else (rows, d)) and got.q.is_contiguous()
        check_codes(got.q, got.scale, v, high, (rows, d, dt, high, transpose))
        # as the product reads it: consecutive rows next to each other
        assert got.scale.t().is_contiguous()
        # the guarded C call writes nothing else
        q, q_ok = guarded(tuple(got.q.shape), torch.uint8, offset=seed % 3)
        s, s_ok = guarded(tuple(got.scale.t().shape), torch.float32)
        xd = x.cuda()
        st = gpu.load().gemm_bt_quantize_blocks(xd.data_ptr(), d, q.data_ptr(), s.data_ptr(), rows, d, high, int(transpose),
                                                {"f32": gpu.F32, "f16": gpu.F16, "bf16": gpu.BF16}[dt], gpu.FP8_E4M3,
                                                torch.cuda.current_stream().cuda_stream)
        assert st == gpu.OK
        q_ok(), s_ok()
        assert torch.equal(q, got.q.view(torch.uint8)) and torch.equal(s.t(), got.scale)


@pytest.mark.gpu
def test_quantize_blocks_layouts(gpu):
    wide = randn(1, 300, 700, dtype=torch.bfloat16).cuda()
    for x in (wide[:, 3:336], wide[::2, 64:397], wide.t()[:333].t()[:, :333], wide[:, 1:257]):
        for high, transpose in itertools.product((1, 128), (False, True)):
            got = gpu.quantize_blocks(x, block=(high, 128), transpose=transpose)
            want = gpu.quantize_blocks(x.contiguous(), block=(high, 128), transpose=transpose)
            assert torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8)) and torch.equal(got.scale, want.scale)
    cube = randn(2, 3, 5, 200).cuda()
    got = gpu.quantize_blocks(cube)
    want = gpu.quantize_blocks(cube.view(15, 200))
    assert got.q.shape == cube.shape and got.scale.shape == (3, 5, 2)
    assert torch.equal(got.scale.reshape(15, 2), want.scale) and torch.equal(got.q.view(torch.uint8).view(15, 200), want.q.view(torch.uint8))
    assert gpu.quantize_blocks(cube[0, 0]).scale.shape == (2,)
    z = torch.zeros(0, 200, device="cuda")
    for x, t, q, s in ((z, False, (0, 200), (0, 2)), (z, True, (200, 0), (200, 0)), (z.t().contiguous(), False, (200, 0), (200, 0))):
        got = gpu.quantize_blocks(x, transpose=t)
        assert got.q.shape == q and got.scale.shape == s


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DT)
def test_quantize_blocks_extremes(gpu, dt):
    """Blocks of zeros, of the type's largest and smallest values, with an infinity or a NaN: each block by itself."""
    big, tiny = torch.finfo(DT[dt]).max, torch.finfo(DT[dt]).smallest_normal
    x = randn(3, 260, 400)
    x[0, :128] = 0.0
    x[1, 5] = float("inf")
    x[2, 399] = float("nan")
    x[3, 128:256] = big
    x[4, 130] = -float("inf")
    x[200, 128:256] = tiny
    x = x.to(DT[dt])
    for high, transpose in itertools.product((1, 128), (False, True)):
        got = gpu.quantize_blocks(x.cuda(), block=(high, 128), transpose=transpose)
        v = (x.t() if transpose else x).double()
        bad = ~torch.isfinite(block_max(torch.where(torch.isfinite(v), 0.0, float("inf")), high))
        assert torch.equal(torch.isnan(got.scale.cpu()), bad), (dt, high, transpose)
        keep = ~bad.repeat_interleave(high, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
        r = torch.where(keep, v, 0.0)
        want = torch.clamp(block_max(r, high) / 448, min=2.0 ** -100)
        s = got.scale.cpu().double()
        assert bool(((s - want).abs()[~bad] <= 2 * u * want[~bad]).all())
        q = got.q.float().double().cpu()[:, :v.shape[1]] * want.repeat_interleave(high, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
        step = want.repeat_interleave(high, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
        assert bool(((q - r).abs()[keep] <= 2.0 ** -4 * r.abs()[keep] * (1 + 16 * u) + 2.0 ** -10 * step[keep]).all()), (dt, high, transpose)


# ------------------------------------------------------------------ the product

def operands(gpu, M, N, K, high, seed):
    """Quantised on the CPU's side of the definition: codes and scales of any values, as strided scales."""
    x = randn(seed, M, K).to(F8)
    w = randn(seed + 1, N, K).to(F8)
    sx = torch.exp(randn(seed + 2, M, up(K, 128)))
    sw = torch.exp(randn(seed + 3, up(N, high), up(K, 128))) * max(K, 1) ** -0.5
    return x, w, sx, sw


def product_tol(x, w, out):
    """Of the sums of x and w (scaled, in 64 bits) for results of type out."""
    tol = (sum_tol if out == torch.float32 else eight_bit_tol)(x, w)
    return tol + (x.shape[1] / 128 + 4) * u * torch.mm(x.abs(), w.abs().t().contiguous())


def strided(t):
    return t.cuda().t().contiguous().t()


def check(gpu, M, N, K, high, outd, act, bias=None, res=None, pre=False, seed=0, offset=0, rowwise=False, **_):
    say("block linear", M, N, K, "rows", high, outd, act, "bias", bias, "res", res, "pre", pre, "seed", seed)
    x, w, sx, sw = operands(gpu, M, N, K, high, seed)
    g = lambda t: None if t is None else t.cuda()
    b = randn(seed + 4, N, dtype=DT[bias]) if bias else None
    r = randn(seed + 5, M, N, dtype=DT[res]) if res else None
    y, untouched = guarded((M, N), DT[outd], offset=offset)
    lay = (lambda t: t.cuda()) if rowwise else strided
    got = gpu.block_linear(x.cuda(), w.cuda(), lay(sx), lay(sw), bias=g(b), activation=act, residual=g(r), out_dtype=DT[outd],
                           save_preact=pre, out=y)
    untouched()
    xd = (x.double() * spread(sx, M, K, 1)).cuda()
    wd = (w.double() * spread(sw, N, K, high)).cuda()
    z = torch.mm(xd, wd.t().contiguous()).cpu()
    tol = product_tol(xd, wd, DT[outd]).cpu()
    if b is not None:
        z = z + b.double()
        tol = tol + u * z.abs()
    if pre:
        assert got[0] is y
        close(got[1], z, tol, "preact")
    a = act64(z, act)
    tol = 1.13 * tol + (0 if act == "none" else 2.0 ** -20 * z.abs())
    if r is not None:
        a = a + r.double()
        tol = tol + u * a.abs()
    close(y, a, tol, "y")


SHAPES = [(1, 1, 16), (520, 4096, 208), (1100, 1500, 400), (4400, 4096, 64), (2100, 4350, 336), (1040, 2000, 144), (1, 72, 4096), (16, 8192, 512), (1, 4104, 4096), (5, 6001, 272), (16, 4099, 8208), (3, 5000, 128), (64, 512, 8192),
          (33, 4096, 4096), (200, 300, 8208), (7, 70, 16384), (129, 1000, 4112), (33, 65, 144), (130, 264, 208), (300, 333, 128),
          (700, 1100, 128), (1000, 2050, 400), (2050, 2050, 64), (2048, 4352, 80), (4100, 4096, 48), (4096, 4097, 32), (1000, 3000, 2064),
          (2048, 4096, 1024), (5000, 3333, 144),
          (16, 12300, 528), (2, 16390, 2064), (13, 32768, 400), (9, 24580, 4112)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("high", [128, 1])
def test_block_linear(gpu, high, shape):
    n = sum(shape)
    for i in (n, n + 1, n + 2):  # one of each type of result
        o = options(i)
        o["bias"] = "bf16" if o["bias"] == "own" else o["bias"]
        check(gpu, *shape, high, seed=n, rowwise=i % 2 == 1, **o)


def test_shapes_cover_every_kernel():
    seen = set()
    for (M, N, K), high, out in itertools.product(SHAPES, (1, 128), (gb.BF16, gb.F32)):
        p = gb.gemm_bt_plan_block(M, N, K, high, out)
        parts = [p] + ([gb.gemm_bt_plan_block(M - p.split_rows, N, K, high, out)] if p.split_rows else [])
        seen |= {(high, out, q.kernel, q.variant, q.split_tiles > 0, p.split_rows > 0) for q in parts}
    for high, out in itertools.product((1, 128), (gb.BF16, gb.F32)):
        kinds = {(k, v, s) for h, o, k, v, s, _ in seen if (h, o) == (high, out)}
        large = {(4, 0, False), (4, 1, False)} if (high, out) != (1, gb.F32) else set()
        widest = {(4, 3, False)} if (high, out) == (128, gb.BF16) else set()
        assert kinds == large | widest | {(4, 2, False), (4, 4, False), (4, 4, True)} | {(3, v, False) for v in (0, 1, 2)}, (high, out, kinds)
    assert {h for h, o, _, _, _, rows in seen if rows} == {1, 128}


@pytest.mark.gpu
def test_every_term_and_empty_sums(gpu):
    for act, outd, high in itertools.product(ACTS, DT, (1, 128)):
        check(gpu, 77, 141, 160, high, outd, act, bias="f16", res="bf16", pre=True, seed=1)
        check(gpu, 9, 4200, 160, high, outd, act, bias="f32", res="f16", pre=True, seed=2)
        check(gpu, 20, 30, 0, high, outd, act, bias="f32", res="f32", pre=True, seed=3)
    z = lambda *s: torch.zeros(*s, device="cuda")
    x, w = z(4, 256).to(F8), z(130, 256).to(F8)
    assert gpu.block_linear(x[:0], w, z(0, 2), z(2, 2)).shape == (0, 130)
    assert gpu.block_linear(x, w[:0], z(4, 2), z(0, 2)).shape == (4, 0)
    assert gpu.block_linear(x.view(2, 2, 256), w, z(2, 2, 2), z(130, 2)).shape == (2, 2, 130)
    assert gpu.block_linear(x[0], w, z(2), z(2, 2)).shape == (130,)


@pytest.mark.gpu
def test_scales_of_extreme_size(gpu):
    """Blocks whose scales are far from 1 and from each other, NaN in one block alone, and infinities."""
    for M, N, K, high in ((40, 300, 640, 128), (9, 4200, 640, 1), (600, 520, 640, 128), (600, 520, 640, 1)):
        x, w, sx, sw = operands(gpu, M, N, K, high, 7)
        sx[1] *= 2.0 ** 40
        sx[2, 1] *= 2.0 ** -60
        sx[3, 4] = float("nan")
        sx[5] = 2.0 ** -100
        sw[:, 2] *= 2.0 ** -30
        row = sw.shape[0] - 1
        sw[row, 0] = float("nan")
        got = gpu.block_linear(x.cuda(), w.cuda(), strided(sx), strided(sw), out_dtype=torch.float32).cpu()
        bad = torch.zeros(M, N, dtype=torch.bool)
        bad[3] = True
        bad[:, row * high:] = True
        assert torch.equal(torch.isnan(got), bad), (M, N, high)
        xd, wd = x.double() * spread(sx, M, K, 1), w.double() * spread(sw, N, K, high)
        xd, wd = torch.nan_to_num(xd), torch.nan_to_num(wd)
        want = xd @ wd.t()
        tol = product_tol(xd, wd, torch.float32)
        assert bool(((got.double() - want).abs() <= tol + u * want.abs() + 2.0 ** -126)[~bad].all()), (M, N, high)


@pytest.mark.gpu
def test_scale_layouts_and_starts(gpu):
    """Scales in any layout, operands off 16-byte boundaries or strided: the same bits."""
    for M, N, K, high in ((70, 300, 640, 128), (9, 4200, 640, 128), (300, 200, 640, 1)):
        x, w, sx, sw = (t.cuda() for t in operands(gpu, M, N, K, high, 11))
        want = gpu.block_linear(x, w, strided(sx), strided(sw))
        assert torch.equal(gpu.block_linear(x, w, sx, sw), want)
        wide = torch.full((M, 13), float("nan"), device="cuda")
        wide[:, 3:13:2] = sx
        assert torch.equal(gpu.block_linear(x, w, wide[:, 3:13:2], sw), want)
        one = sx[:1].expand(M, -1)  # one row of scales for all
        assert torch.equal(gpu.block_linear(x, w, one, sw), gpu.block_linear(x, w, one.contiguous(), sw))
        moved = torch.empty(x.numel() + 3, dtype=torch.uint8, device="cuda")
        moved[3:] = x.view(torch.uint8).flatten()
        assert torch.equal(gpu.block_linear(moved[3:].view(F8).view(M, K), w, sx, sw), want)
        assert torch.equal(gpu.block_linear(x, w.t().contiguous().t(), sx, sw), want)
        out = torch.empty_like(want)
        r = randn(3, M, N, dtype=torch.bfloat16).cuda()
        there = r.clone()
        a = gpu.block_linear(x, w, sx, sw, residual=r, out=out)
        assert a is out and torch.equal(gpu.block_linear(x, w, sx, sw, residual=there, out=there), out)


@pytest.mark.gpu
def test_training_step_in_8_bits(gpu):
    """y = x W^T, dx = dy W and dW = dy^T x, each from blocks along its own sum, against 64 bits of the values in blocks."""
    for M, N, K in ((130, 264, 528), (37, 144, 272), (1000, 512, 1024)):
        say("training step", M, N, K)
        x, w, dy = (randn(i, *s, dtype=torch.bfloat16).cuda() for i, s in enumerate(((M, K), (N, K), (M, N))))
        value = lambda t, rows, cols, high: (t.q.float().double().cpu()[:, :cols] * spread(t.scale, rows, cols, high)).cuda()
        # forward; then dx sums over N, dW over M
        for a, b, rows, cols, depth, high in (
                (gpu.quantize_blocks(x), gpu.quantize_blocks(w, block=(128, 128)), M, N, K, 128),
                (gpu.quantize_blocks(dy), gpu.quantize_blocks(w, block=(128, 128), transpose=True), M, K, N, 128),
                (gpu.quantize_blocks(dy, transpose=True), gpu.quantize_blocks(x, transpose=True), N, K, M, 1)):
            qa = a.q
            if b.q.shape[1] != qa.shape[1]:  # (a weight's rows transposed are filled up to a multiple of 16)
                qa = torch.nn.functional.pad(qa.view(torch.uint8), (0, b.q.shape[1] - qa.shape[1])).view(F8)
            got = gpu.block_linear(qa, b.q, a.scale, b.scale, out_dtype=torch.float32)
            av, bv = value(a, rows, depth, 1), value(b, cols, depth, high)
            want = torch.mm(av, bv.t().contiguous())
            tol = product_tol(av, bv, torch.float32)
            close(got, want.cpu(), tol.cpu(), (M, N, K, rows, cols))
        # and from the 16-bit values themselves: each code within 2^-4 of its value, or half the smallest step of its block
        q = gpu.quantize_blocks(x)
        off = (value(q, M, K, 1) - x.double()).abs()
        s = spread(q.scale, M, K, 1).cuda()
        assert bool((off <= 2.0 ** -4 * x.double().abs() * (1 + 8 * u) + 2.0 ** -10 * s).all())


@pytest.mark.gpu
def test_large_offsets(gpu):
    """Results past 2^31 bytes from their start, and scales of 270000 rows."""
    M, N, K = 270000, 4100, 144
    say("block linear", M, N, K)
    x = torch.randint(0, 100, (M, K), dtype=torch.uint8, device="cuda").view(F8)
    w = torch.randint(0, 100, (N, K), dtype=torch.uint8, device="cuda").view(F8)
    sx = torch.rand(2, M, device="cuda").t() + 0.5
    sw = torch.rand(2, up(N, 128), device="cuda").t() + 0.5
    sx, sw = sx.t().contiguous().t(), sw.t().contiguous().t()
    y = gpu.block_linear(x, w, sx, sw)
    wd = w.double().cpu() * spread(sw, N, K, 128)
    for rows in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        xd = x[rows].double().cpu() * spread(sx[rows], 300, K, 1)
        close(y[rows], xd @ wd.t(), product_tol(xd, wd, y.dtype), "y")


@pytest.mark.gpu
def test_streams_and_graphs(gpu):
    """Quantisation and products, a split one among them, on side streams and in replayed graphs."""
    M, N, K = 64, 512, 8192
    assert gpu.gemm_bt_plan_block(M, N, K, 128, gpu.BF16).split_tiles > 0
    make = lambda seed: [randn(seed, M, K, dtype=torch.bfloat16).cuda(), randn(seed + 1, N, K, dtype=torch.bfloat16).cuda()]

    def both(x, w, stream=None):
        a = gpu.quantize_blocks(x, stream=stream)
        b = gpu.quantize_blocks(w, block=(128, 128), stream=stream)
        return [a.q.view(torch.uint8), a.scale, gpu.block_linear(a.q, b.q, a.scale, b.scale, activation="silu", stream=stream)]
    sets = make(1), make(11)
    want = [both(*s) for s in sets]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        got = both(*sets[0], stream=handle)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    fed = [t.clone() for t in sets[0]]
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(both(*fed))
    for i, which in ((0, 0), (1, 1), (0, 1), (1, 0)):
        for t, v in zip(fed, sets[i]):
            t.copy_(v)
        graphs[which].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[which], want[i])), (i, which)
        assert all(torch.equal(a, b) for a, b in zip(both(*sets[1 - i]), want[1 - i]))


# ------------------------------------------------------------------ refusals

def quant(x=16, ldx=8, q=16, scale=16, rows=2, d=8, high=1, transpose=0, xt=gb.BF16, qt=gb.FP8_E4M3):
    return int(gb.load().gemm_bt_quantize_blocks(x, ldx, q, scale, rows, d, high, transpose, xt, qt, None))


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), BAD), (dict(d=-1), BAD), (dict(high=2), BAD), (dict(high=0), BAD), (dict(transpose=2), BAD), (dict(xt=gb.INT8), UNSUP),
    (dict(qt=gb.INT8), UNSUP), (dict(qt=gb.FP8_E5M2), UNSUP), (dict(rows=2 ** 31 + 1), UNSUP), (dict(d=2 ** 26 + 1, ldx=2 ** 27), UNSUP),
    (dict(x=None), BAD), (dict(q=None), BAD), (dict(scale=None), BAD), (dict(x=17), BAD), (dict(scale=18), BAD), (dict(ldx=7), BAD),
    (dict(rows=0, x=None, q=None, scale=None), gb.OK), (dict(d=0, x=None, q=None, scale=None), gb.OK),
])
def test_quantize_refusals(kw, want):
    assert quant(**kw) == want


def block(A=16, B=16, C=16, M=4, N=4, K=16, sa=16, ra=1, ba=4, sb=16, rb=1, bb=1, high=128, i=gb.FP8_E4M3, o=gb.BF16, ws=None, n=0, **terms):
    from dense_tiled_gemm_amd.layers import Epilogue

    return int(gb.load().gemm_bt_block(A, B, C, M, N, K, sa, ra, ba, sb, rb, bb, high, i, o, ctypes.byref(Epilogue(**terms)), ws, n, None))


@pytest.mark.parametrize("kw,want", [
    (dict(i=gb.FP8_E5M2), UNSUP), (dict(i=gb.BF16), UNSUP), (dict(i=gb.INT8), UNSUP), (dict(o=gb.INT32), UNSUP), (dict(o=gb.FP8_E4M3), UNSUP),
    (dict(K=8), UNSUP), (dict(K=120), UNSUP), (dict(A=8), UNSUP), (dict(B=24), UNSUP), (dict(high=64), BAD), (dict(M=-1), BAD),
    (dict(N=-1), BAD), (dict(K=-16), BAD), (dict(C=None), BAD), (dict(C=17), BAD), (dict(C=18, o=gb.F32), BAD), (dict(A=None), BAD),
    (dict(B=None), BAD), (dict(sa=None), BAD), (dict(sb=None), BAD), (dict(sa=18), BAD), (dict(sb=17), BAD), (dict(ra=-1), BAD),
    (dict(bb=-1), BAD), (dict(ra=1 << 20), UNSUP), (dict(rb=1 << 20), UNSUP), (dict(ba=1 << 26), UNSUP), (dict(bb=1 << 26), UNSUP),
    (dict(K=1 << 23), UNSUP), (dict(N=1 << 23), UNSUP), (dict(M=1 << 31), UNSUP), (dict(activation=9), BAD),
    (dict(bias=17, bias_dtype=gb.BF16), BAD), (dict(residual=16, residual_dtype=gb.INT32), BAD),
    (dict(M=0, A=None, B=None, C=None, sa=None, sb=None), gb.OK), (dict(N=0, A=None, B=None, C=None, sa=None, sb=None), gb.OK),
])
def test_refusals(kw, want):
    assert block(**kw) == want


def test_workspaces_and_plans():
    lib, n = gb.load(), ctypes.c_size_t()
    f = lib.gemm_bt_block_workspace_size
    assert f(4, 4, 16, 1, gb.BF16, None) == BAD and f(-1, 4, 16, 1, gb.BF16, ctypes.byref(n)) == BAD
    assert f(4, 4, 8, 1, gb.BF16, ctypes.byref(n)) == UNSUP and f(4, 4, 16, 64, gb.BF16, ctypes.byref(n)) == BAD
    assert f(4, 4, 16, 1, gb.INT32, ctypes.byref(n)) == UNSUP and n.value == 0
    assert f(64, 512, 8192, 128, gb.BF16, ctypes.byref(n)) == gb.OK
    p = gb.gemm_bt_plan_block(64, 512, 8192, 128, gb.BF16)
    assert n.value == p.workspace_bytes == 16384 + p.grid * 64 * 64 * 4 and p.grid == p.split_tiles * 4
    assert block(M=64, N=512, K=8192, ba=64, ws=16, n=n.value - 1) in (BAD, gb.ERR_NO_DEVICE)  # (checked after the device)
    assert lib.gemm_bt_plan_block(4, 4, 16, 1, gb.BF16, 16, 16, None) == BAD


def test_wrappers_check_before_the_library():
    x, s = torch.zeros(2, 16).to(F8), torch.zeros(2, 1)
    for call in (lambda: gb.quantize_blocks(s), lambda: gb.block_linear(x, x, s, s)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_wrapper_refusals(gpu):
    z = lambda *s: torch.zeros(*s, device="cuda")
    x, w, sx, sw = z(4, 256).to(F8), z(130, 256).to(F8), z(4, 2), z(2, 2)
    for error, call in ((ValueError, lambda: gpu.quantize_blocks(sx, block=(128, 1))), (TypeError, lambda: gpu.quantize_blocks(sx, dtype=torch.int8)),
                        (TypeError, lambda: gpu.quantize_blocks(x)), (ValueError, lambda: gpu.quantize_blocks(z(()))),
                        (TypeError, lambda: gpu.block_linear(sx, w, sx, sw)), (TypeError, lambda: gpu.block_linear(x, w.to(torch.float8_e5m2), sx, sw)),
                        (ValueError, lambda: gpu.block_linear(x, w[:, :128], sx, sw)), (ValueError, lambda: gpu.block_linear(x, w, z(4, 3), sw)),
                        (ValueError, lambda: gpu.block_linear(x, w, z(3, 2), sw)), (ValueError, lambda: gpu.block_linear(x, w, sx.half(), sw)),
                        (ValueError, lambda: gpu.block_linear(x, w, sx, z(3, 2))), (ValueError, lambda: gpu.block_linear(x, w, sx, z(2, 3))),
                        (ValueError, lambda: gpu.block_linear(x, w, sx, sw, bias=z(4))), (TypeError, lambda: gpu.block_linear(x, w, sx, sw, out_dtype=F8)),
                        (gpu.GemmBtError, lambda: gpu.block_linear(x[:, :120], w[:, :120], z(4, 1), z(2, 1)))):
        with pytest.raises(error):
            call()


@pytest.mark.gpu
def test_codes_without_a_value(gpu):
    """A NaN among the codes reaches its own row or column of the product, for every kind of result."""
    for (M, N, K, high), dt in itertools.product(((40, 300, 656, 128), (9, 4200, 640, 1), (600, 520, 640, 128)),
                                                 (torch.bfloat16, torch.float32)):
        x, w, sx, sw = operands(gpu, M, N, K, high, 19)
        xb, wb = x.view(torch.uint8).clone(), w.view(torch.uint8).clone()
        xb[3, 5], xb[M - 1, K - 1], wb[7, 200] = 0x7F, 0xFF, 0x7F
        got = gpu.block_linear(xb.view(F8).cuda(), wb.view(F8).cuda(), sx.cuda(), sw.cuda(), out_dtype=dt).cpu()
        bad = torch.zeros(M, N, dtype=torch.bool)
        bad[3] = bad[M - 1] = True
        bad[:, 7] = True
        assert torch.equal(torch.isnan(got), bad), (M, N, high, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(1, 128), (5, 100), (130, 300), (300, 1024)])
def test_codes_are_rounded_once(gpu, rows, d):
    """16-bit inputs: the codes are those of v / scale exactly.  v 448 / amax is a quotient of two integers, the divisor
    below 2^11: on the edge between two codes, or further from it than 2^-17 of itself, so fp32 holds it on the right side."""
    for dt, high, transpose in itertools.product((torch.bfloat16, torch.float16), (1, 128), (False, True)):
        say("block codes", rows, d, dt, high, transpose)
        x = randn(rows + d, rows, d, std=3.0).to(dt)
        v = (x.t() if transpose else x).double()
        full = spread(block_max(v, high), *v.shape, high)
        want = (v * 448 / full).float().to(F8)
        got = gpu.quantize_blocks(x.cuda(), block=(high, 128), transpose=transpose).q.cpu()[:, :v.shape[1]]
        assert torch.equal(got.float(), want.float()), (rows, d, dt, high, transpose)


def codes64(v):
    """v in E4M3, to nearest even, and how far v is from the edge between two codes, in steps."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    t = v / step
    return torch.round(t) * step, (t - t.floor() - 0.5).abs()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(130, 300), (1000, 4096)])
def test_codes_of_fp32_are_rounded_once(gpu, rows, d):
    """fp32 inputs: the codes are those of v 448 / amax unless it lies within 2^-40 of a code's edge.  What is left out of
    448 / amax and of the product in two parts is below 2^-45 of it; a rounding to fp32 before would change 1 in 3e6."""
    for high, transpose in itertools.product((1, 128), (False, True)):
        say("block codes fp32", rows, d, high, transpose)
        x = randn(rows + d, rows, d, std=3.0)
        v = (x.t() if transpose else x).double()
        full = spread(block_max(v, high), *v.shape, high)
        want, edge = codes64(v * 448 / full)
        got = gpu.quantize_blocks(x.cuda(), block=(high, 128), transpose=transpose).q.cpu()[:, :v.shape[1]].float().double()
        assert bool(((got == want) | (edge < 2.0 ** -36)).all()), (rows, d, high, transpose, int((got != want).sum()))
