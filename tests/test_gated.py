"""The gated product and its backward pass against plain implementations in 64 bits.

Where the tolerances come from (u = 2^-24): a sum of K terms is within K u of the sum of their magnitudes in any order (int8:
exact, then rounded once; 8-bit floats: see eight_bit_tol); scales and bias are three and one roundings more, so that Zg and Zu are each known to T; the
activation is no steeper than 1.13 and within 2^-20 |z| of itself; the product of a = act(Zg), known to A, and Zu is within
A |Zu| + (|a| + A) T + u |a Zu|; then one rounding into the stored type.  dz is rounded into the inputs' 16-bit type before
the backward products, its slope within 2^-20 (1 + |z|^3) and its activation within 2^-20 |z| before that.
"""
import ctypes
import itertools

import pytest
import torch

import dense_tiled_gemm_amd as gb
from test_layers_gpu import ACTS, DT, SHAPES16, TINY, UNIT, act64, close, gen, guarded, options, randn, say, slope64, u

BAD, UNSUP = gb.ERR_INVALID_VALUE, gb.ERR_UNSUPPORTED
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
CODE = {"bf16": gb.BF16, "f16": gb.F16, "e4m3": gb.FP8_E4M3, "e5m2": gb.FP8_E5M2, "i8": gb.INT8}

# the same tile shapes with 2 N columns
SHAPES = [(M, (N + 1) // 2, K) for M, N, K in SHAPES16] + [(16, 4097, 2048), (16, 6150, 1031), (3, 8195, 2056), (7, 16384, 200), (11, 12290, 4096), (33, 7, 40), (1, 3, 8), (300, 5, 72)]


def inputs(M, N, K, ind, seed):
    if ind == "i8":
        return tuple(torch.randint(-128, 128, s, generator=gen(seed + i), dtype=torch.int8) for i, s in enumerate(((M, K), (2 * N, K))))
    t = F8.get(ind) or DT[ind]
    return randn(seed, M, K).to(t), randn(seed + 1, 2 * N, K, std=K ** -0.5 if K else 1.0).to(t)


def sum_tol(x, w):
    """How far a product's fp32 sums of x and w (in 64 bits) may be off: K roundings in any order."""
    mag = torch.mm(x.abs(), w.abs().t().contiguous())
    return x.shape[1] * u * mag


def eight_bit_tol(x, w):
    """The same for 8-bit floats.

    The matrix instructions add 8-bit floats in groups of 8 consecutive k.  Within a group each product is cut, towards
    zero, to a multiple of 2^(E - 13), E the largest sum of a pair's exponents (test_products_of_8_bit_floats): the largest
    one stays whole, each of the 7 others loses less than 2^-13 of it, which is at most the product of both groups' largest
    magnitudes.  The groups' sums are added in fp32 like any other terms.
    """
    top = lambda t: torch.nn.functional.pad(t.abs(), (0, -t.shape[1] % 8)).unflatten(1, (-1, 8)).amax(2)
    return sum_tol(x, w) + 7 * 2.0 ** -13 * torch.mm(top(x), top(w).t().contiguous())


@pytest.mark.gpu
def test_products_of_8_bit_floats(gpu):
    """Sums of 2^16 and one other term, near it and far from it in k, in the tiled and in the streaming kernel."""
    for t, (M, N) in itertools.product(F8.values(), ((64, 64), (1, 4104))):
        x, w = torch.zeros(M, 64), torch.zeros(N, 64)
        x[:, 0] = w[:, 0] = 256.0
        for at, small in itertools.product((1, 7, 8, 63), (256.0, 28.0, 12.0, 8.0, 4.0, 1.0, -28.0, -12.0, -4.0)):
            x[:, 1:], w[:, 1:] = 0.0, 0.0
            x[:, at], w[:, at] = small, 1.0
            got = gpu.linear(x.to(t).cuda(), w.to(t).cuda(), out_dtype=torch.float32).cpu()
            quantum = 8.0 if at < 8 else 2.0 ** -7
            want = 65536.0 + int(float(x.to(t)[0, at]) / quantum) * quantum
            assert bool((got == want).all()), (t, M, at, small, float(got[0, 0]), want)


def check(gpu, M, N, K, ind, outd, act, bias=None, pre=False, scales=False, seed=0, offset=0, **_):
    say("gated", M, N, K, ind, outd, act, "bias", bias, "pre", pre, "scales", scales, "seed", seed)
    x, w = inputs(M, N, K, ind, seed)
    g = lambda t: None if t is None else t.cuda()
    b = randn(seed + 2, 2 * N, dtype=DT[bias]) if bias else None
    xs = torch.rand(M, generator=gen(seed + 4)) + 0.5 if scales else None
    ws = (torch.rand(2 * N, generator=gen(seed + 5)) + 0.5) * (1 / (74 * 74 * max(K, 1) ** 0.5) if ind == "i8" else 1) if scales else None
    y, untouched = guarded((M, N), DT[outd], offset=offset)
    got = gpu.gated_linear(x.cuda(), w.cuda(), bias=g(b), activation=act, x_scale=g(xs), weight_scale=g(ws), out=y, out_dtype=DT[outd],
                           save_preact=pre)
    untouched()
    x64, w64 = x.float().double().cuda(), w.float().double().cuda()
    z = torch.mm(x64, w64.t().contiguous()).cpu()
    tol = u * z.abs() if ind == "i8" else (eight_bit_tol(x64, w64) if ind in F8 else sum_tol(x64, w64)).cpu()
    if scales:
        scale = xs.double()[:, None] * ws.double()
        z, tol = z * scale, tol * scale
        tol = tol + 3 * u * z.abs()
    if b is not None:
        z = z + b.double()
        tol = tol + u * z.abs()
    if pre:
        assert got[0] is y
        close(got[1], z, tol, "preact")
    gate, up, tg, tu = z[:, :N], z[:, N:], tol[:, :N], tol[:, N:]
    a = act64(gate, act)
    ta = 1.13 * tg + (0 if act == "none" else 2.0 ** -20 * gate.abs())
    close(y, a * up, ta * up.abs() + (a.abs() + ta) * tu + 2 * u * (a * up).abs(), "y")
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("n,shape", list(enumerate(SHAPES)))
def test_gated_shapes(gpu, n, shape):
    for i in (n, n + 7):
        ind = ("bf16", "f16")[(n + i) % 2]
        o = options(i)
        o["bias"] = ind if o["bias"] == "own" else o["bias"]
        check(gpu, *shape, ind, seed=n, **o)


def test_shapes_cover_every_kernel():
    seen = set()
    for M, N, K in SHAPES:
        p = gb.gemm_bt_plan_epi(M, 2 * N, K, gb.BF16, gb.F32)
        parts = [p] + ([gb.gemm_bt_plan_epi(M - p.split_rows, 2 * N, K, gb.BF16, gb.F32)] if p.split_rows else [])
        seen |= {(q.kernel, q.variant, q.split_tiles > 0) for q in parts}
    assert {v for k, v, s in seen if k == 4 and not s} == {0, 1, 2, 6, 7, 8, 9, 12, 13, 14, 15}, seen
    assert {v for k, v, s in seen if k == 4 and s} == {1, 10, 11, 12}, seen
    assert any(k == 3 for k, _, _ in seen)


@pytest.mark.gpu
@pytest.mark.parametrize("ind", ["e4m3", "e5m2", "i8"])
@pytest.mark.parametrize("shape", [(1, 1, 16), (1, 36, 4096), (33, 33, 144), (130, 132, 208), (700, 550, 128), (2050, 1025, 64),
                                   (2048, 2176, 80), (4100, 2048, 48), (16, 4096, 512), (1, 2052, 4096), (5, 3001, 272), (64, 256, 8192),
                                   (33, 2048, 4096), (7, 35, 16384), (4352, 2048, 64), (16, 6150, 1040), (3, 8195, 2064), (7, 16384, 208)])
def test_gated_eight_bits(gpu, ind, shape):
    n = sum(shape)
    for i in (n, n + 5):
        o = options(i)
        o["bias"] = "bf16" if o["bias"] == "own" else o["bias"]
        o["scales"] = ind == "i8" or i % 2 == 0
        check(gpu, *shape, ind, seed=n, **o)


@pytest.mark.gpu
def test_every_term(gpu):
    for act, outd in itertools.product(ACTS, DT):
        check(gpu, 77, 71, 96, "bf16", outd, act, bias="f16", pre=True, seed=1)
        check(gpu, 9, 3001, 96, "f16", outd, act, bias="bf16", pre=True, scales=True, seed=2)
        check(gpu, 20, 30, 0, "bf16", outd, act, bias="f32", pre=True, seed=3)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    assert gpu.gated_linear(z(0, 16), z(8, 16)).shape == (0, 4)
    assert gpu.gated_linear(z(3, 16), z(0, 16)).shape == (3, 0)
    assert gpu.gated_linear(z(2, 4, 16), z(8, 16), save_preact=True)[1].shape == (2, 4, 8)
    assert gpu.gated_linear(z(16), z(8, 16)).shape == (4,)


@pytest.mark.gpu
def test_strided_inputs_and_starts(gpu):
    """Columns of wider tensors, a transposed weight, tensors off 16-byte boundaries: the same bits as from dense ones."""
    x, w = randn(1, 70, 96, dtype=torch.bfloat16).cuda(), randn(2, 60, 96, std=0.1, dtype=torch.bfloat16).cuda()
    want = gpu.gated_linear(x, w)
    wide = torch.zeros(70, 101, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:98] = x
    assert torch.equal(gpu.gated_linear(wide[:, 2:98], w.t().contiguous().t()), want)
    for t in (torch.bfloat16, torch.float8_e4m3fn, torch.int8):
        a, b = (v.float().mul(8).round().to(t) for v in (x, w))
        want = gpu.gated_linear(a, b)
        moved = []
        for v in (a, b):
            buf = torch.empty(v.numel() + 1, dtype=t, device="cuda")
            buf[1:].copy_(v.flatten())
            moved.append(buf[1:].view(v.shape))
        got = gpu.gated_linear(*moved)
        assert torch.equal(got, want)  # whole numbers: every sum is exact in any order


@pytest.mark.gpu
def test_large_offsets(gpu):
    """Results and pre-activations past 2^31 bytes from their start."""
    M, N, K = 270000, 2050, 32
    say("gated", M, N, K)
    x, w = randn(1, M, K, dtype=torch.bfloat16).cuda(), randn(2, 2 * N, K, dtype=torch.bfloat16).cuda()
    y, z = gpu.gated_linear(x, w, activation="relu", save_preact=True)
    for rows in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        z64 = x[rows].double().cpu() @ w.double().cpu().t()
        tol = K * u * (x[rows].double().cpu().abs() @ w.double().cpu().abs().t())
        close(z[rows], z64, tol, "preact")
        a, up = z64[:, :N].clamp_min(0), z64[:, N:]
        close(y[rows], a * up, tol[:, :N] * up.abs() + (a + tol[:, :N]) * tol[:, N:] + u * (a * up).abs(), "y")


@pytest.mark.gpu
def test_non_finite(gpu):
    """Infinities and NaN stay in their rows and columns."""
    M, N, K = 40, 35, 64
    x, w, b = randn(1, M, K), randn(2, 2 * N, K, std=0.1), randn(3, 2 * N)
    x[3, 5] = float("nan")
    w[9, 0] = float("nan")       # a gate's row
    w[N + 11, 0] = float("inf")  # a row of the other factor
    b[7] = float("inf")
    x, w = x.bfloat16(), w.bfloat16()
    for act in ACTS:
        y = gpu.gated_linear(x.cuda(), w.cuda(), bias=b.cuda(), activation=act, out_dtype=torch.float32).cpu()
        rows = torch.arange(M) != 3
        assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[:, 9]).all())
        cols = torch.ones(N, dtype=torch.bool)
        cols[[7, 9, 11]] = False
        assert bool(torch.isfinite(y[rows][:, cols]).all()), act
        assert bool(torch.isinf(y[rows][:, 7]).all()), act


# ------------------------------------------------------------------ backward

def check_backward(gpu, M, N, K, dt, act, bias=True, seed=0):
    say("gated backward", M, N, K, dt, act, "seed", seed)
    x, w = randn(seed, M, K, dtype=DT[dt]), randn(seed + 1, 2 * N, K, std=max(K, 1) ** -0.5, dtype=DT[dt])
    dy, z = randn(seed + 2, M, N, std=0.1, dtype=DT[dt]), randn(seed + 3, M, 2 * N, std=1.5, dtype=DT[dt])
    got = gpu.gated_linear_backward(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), activation=act, bias_grad=bias)
    x, w, dy = (t.double().cuda() for t in (x, w, dy))
    gate, up = z[:, :N].double(), z[:, N:].double().cuda()
    slope, value, gate = slope64(gate, act).cuda(), act64(gate, act).cuda(), gate.cuda()
    dz = torch.cat((dy * up * slope, dy * value), 1)
    # before the rounding of dz: the activation's part, and three and two roundings of products
    rel = 0 if act == "none" else 2.0 ** -20
    raw = torch.cat((dy.abs() * up.abs() * rel * (1 + gate.abs() ** 3), dy.abs() * rel * gate.abs()), 1) + 3 * u * dz.abs()
    dz_tol = raw + UNIT[DT[dt]] * (dz.abs() + raw) + TINY[DT[dt]]
    size = dz.abs() + dz_tol
    close(got.dx, (dz @ w).cpu(), (dz_tol @ w.abs() + 2 * N * u * (size @ w.abs())).cpu(), "dx")
    close(got.dweight, torch.mm(dz.t().contiguous(), x).cpu(),
          (torch.mm(dz_tol.t().contiguous(), x.abs()) + M * u * torch.mm(size.t().contiguous(), x.abs())).cpu(), "dw")
    if bias:
        close(got.dbias, dz.sum(0).cpu(), (raw.sum(0) + (M + 8) * u * dz.abs().sum(0)).cpu(), "db")
    else:
        assert got.dbias is None


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 4, 8), (5, 32, 72), (17, 4, 512), (100, 128, 264), (333, 500, 520), (1000, 256, 2048), (2049, 512, 72),
                                   # rows that are not whole 16-byte chunks: every remainder of N, and of K
                                   (1, 1, 1), (33, 9, 7), (64, 50, 130), (200, 1001, 64), (77, 515, 40), (50, 12, 24), (19, 13, 16), (40, 30, 8),
                                   (200, 31, 1001), (9, 6, 16), (9, 7, 16), (9, 5, 8), (511, 1025, 333),
                                   # 256 x 256 tiles; sums cut into slices
                                   (2048, 1024, 2050), (4096, 2048, 128), (5000, 32, 200), (70, 2500, 136), (9000, 257, 520), (40000, 260, 512)])
def test_backward(gpu, M, N, K):
    for i, (dt, act) in enumerate(itertools.product(("bf16", "f16"), ACTS)):
        if (M + i) % 2 == 0 and (M * N * K < 5e7 or i in (1, 2, 8)) or M < 100:
            check_backward(gpu, M, N, K, dt, act, bias=i % 3 != 0, seed=M + i)


@pytest.mark.gpu
def test_backward_does_not_read_what_lies_behind_dz(gpu):
    """Rows of dz that are not whole chunks, in a workspace full of NaN."""
    lib = gpu.load()
    for N in (1, 3, 5, 6, 7, 13, 14, 15, 517, 1001):
        M, K = 37, 24
        dy, x, w, z = (randn(i, *s, dtype=torch.bfloat16).cuda() for i, s in enumerate(((M, N), (M, K), (2 * N, K), (M, 2 * N))))
        want = gpu.gated_linear_backward(dy, x, w, z)
        need = ctypes.c_size_t()
        assert lib.gemm_bt_gated_backward_workspace(M, N, K, 4, ctypes.byref(need)) == gpu.OK
        ws = torch.full((need.value,), 0xFF, dtype=torch.uint8, device="cuda")
        out = [torch.full_like(t, float("nan")) for t in want]
        call = lambda n: lib.gemm_bt_gated_backward(dy.data_ptr(), x.data_ptr(), w.data_ptr(), z.data_ptr(), *(t.data_ptr() for t in out),
                                                    M, N, K, 4, gpu.BF16, gpu.BF16, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        assert call(need.value - 1) == BAD
        assert call(need.value) == gpu.OK
        for a, b in zip(out, want):
            assert bool(torch.isfinite(a).all()) and torch.equal(a, b), N


@pytest.mark.gpu
def test_backward_parts_and_places(gpu):
    for M, N, K in ((70, 48, 130), (300, 256, 256), (5000, 32, 200)):
        dy, x, w, z = (randn(i, *s, std=0.3, dtype=torch.bfloat16).cuda() for i, s in enumerate(((M, N), (M, K), (2 * N, K), (M, 2 * N))))
        whole = gpu.gated_linear_backward(dy, x, w, z)
        again = gpu.gated_linear_backward(dy, x, w, z)
        assert all(torch.equal(a, b) for a, b in zip(whole, again))
        for i, kw in enumerate((dict(bias_grad=False, need_dweight=False), dict(bias_grad=False, need_dx=False),
                                dict(need_dx=False, need_dweight=False))):
            part = gpu.gated_linear_backward(dy, x, w, z, **kw)
            assert torch.equal(part[i], whole[i]) and [g is None for g in part] == [j != i for j in range(3)]
        off = []
        for t in (dy, x, w, z):
            buf = torch.zeros(t.numel() + 3, dtype=t.dtype, device="cuda")
            buf[3:] = t.flatten()
            off.append(buf[3:].view(t.shape))
        assert all(torch.equal(a, b) for a, b in zip(whole, gpu.gated_linear_backward(*off)))
        cube = gpu.gated_linear_backward(dy.view(2, M // 2, N), x.view(2, M // 2, K), w, z.view(2, M // 2, 2 * N))
        assert cube.dx.shape == (2, M // 2, K) and torch.equal(cube.dx.view(M, K), whole.dx) and torch.equal(cube.dweight, whole.dweight)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    empty = gpu.gated_linear_backward(z(0, 4), z(0, 16), z(8, 16), z(0, 8))
    assert empty.dx.shape == (0, 16) and not bool(empty.dweight.any()) and not bool(empty.dbias.any())


@pytest.mark.gpu
def test_gradient_against_differences(gpu):
    """dx, dw, db of sum(y * dy) along random directions against central differences of the 64-bit forward pass."""
    M, N, K, step = 6, 10, 24, 1e-5
    x, w, dy, b = (randn(50 + i, *s, dtype=torch.bfloat16) for i, s in enumerate(((M, K), (2 * N, K), (M, N), (2 * N,))))
    w = (w * 0.25).bfloat16()
    for act in ACTS[2:]:
        _, z = gpu.gated_linear(x.cuda(), w.cuda(), bias=b.cuda(), activation=act, save_preact=True)
        got = gpu.gated_linear_backward(dy.cuda(), x.cuda(), w.cuda(), z, activation=act)

        def loss(x, w, b):
            t = x @ w.t() + b
            return float((act64(t[:, :N], act) * t[:, N:] * dy.double()).sum())
        args = [x.double(), w.double(), b.double()]
        for i, grad in enumerate(got):
            v = randn(70 + i, *grad.shape).double()
            move = lambda s: [a + s * v if j == i else a for j, a in enumerate(args)]
            want = (loss(*move(step)) - loss(*move(-step))) / (2 * step)
            along = float((grad.double().cpu() * v).sum())
            # z is kept in 16 bits (its slope no steeper than 1.2, times the other factor), dz and the result are rounded:
            # each entry of the gradient within 4 roundings of 2^-8 of what its terms' magnitudes sum to
            mag = dy.double().abs().max() * 8 * (args[1].abs().sum(0).max() if i == 0 else args[0].abs().sum(0).max() if i == 1 else M)
            assert abs(along - want) <= 4 * 2.0 ** -8 * float(mag) * float(v.square().sum().sqrt()), (act, i, along, want)


@pytest.mark.gpu
def test_streams_and_graphs(gpu):
    """A captured forward and backward pass, a split product among them, replayed with other inputs and eager calls in between."""
    M, N, K = 200, 128, 8192
    assert gpu.gemm_bt_plan_epi(M, 2 * N, K, gpu.BF16, gpu.BF16).split_tiles > 0
    make = lambda seed: [randn(seed, M, K, dtype=torch.bfloat16).cuda(), randn(seed + 1, 2 * N, K, std=0.02, dtype=torch.bfloat16).cuda(),
                         randn(seed + 2, 2 * N, dtype=torch.bfloat16).cuda(), randn(seed + 3, M, N, dtype=torch.bfloat16).cuda()]

    def both(x, w, b, dy, stream=None):
        y, z = gpu.gated_linear(x, w, bias=b, save_preact=True, stream=stream)
        return [y, z, *gpu.gated_linear_backward(dy, x, w, z, stream=stream)]
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

def gated(A=16, B=16, C=16, M=4, N=4, K=16, i=gb.BF16, o=gb.BF16, ws=None, ws_bytes=0, **terms):
    from dense_tiled_gemm_amd.layers import Epilogue

    return int(gb.load().gemm_bt_gated(A, B, C, M, N, K, i, o, ctypes.byref(Epilogue(**terms)), ws, ws_bytes, None))


@pytest.mark.parametrize("kw,want", [
    (dict(o=gb.INT32), UNSUP), (dict(o=gb.FP8_E4M3), UNSUP), (dict(i=gb.F32), UNSUP), (dict(i=gb.INT8, K=131088), UNSUP),
    (dict(i=gb.FP8_E4M3, K=8), UNSUP), (dict(activation=-1), BAD), (dict(activation=5), BAD), (dict(bias=16, bias_dtype=gb.INT8), BAD),
    (dict(bias=17, bias_dtype=gb.BF16), BAD), (dict(residual=16, residual_dtype=gb.BF16), BAD), (dict(preact=18, preact_dtype=gb.F32), BAD),
    (dict(row_scale=18), BAD), (dict(col_scale=2), BAD), (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(N=1 << 30), UNSUP), (dict(C=None), BAD),
    (dict(C=17), BAD), (dict(C=18, o=gb.F32), BAD), (dict(A=None), BAD), (dict(B=None), BAD), (dict(i=gb.FP8_E4M3, A=17), UNSUP),
    (dict(N=(1 << 21) - 1), UNSUP),  # rows of 2 N fp32 past what 256 of them may span
    (dict(M=0, A=None, B=None, C=None), gb.OK), (dict(N=0, A=None, B=None, C=None), gb.OK),
])
def test_refusals(kw, want):
    if kw.get("N") == (1 << 21) - 1:
        kw = dict(kw, o=gb.F32)
    assert gated(**kw) == want


def back(dy=16, x=16, w=16, z=16, dx=16, dw=16, db=16, M=4, N=8, K=8, act=1, t=gb.BF16, zt=gb.BF16, ws=16, nbytes=1 << 30):
    return int(gb.load().gemm_bt_gated_backward(dy, x, w, z, dx, dw, db, M, N, K, act, t, zt, ws, nbytes, None))


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=-1), BAD), (dict(act=9), BAD), (dict(t=gb.F32), UNSUP), (dict(zt=gb.INT8), UNSUP),
    (dict(zt=gb.INT8, act=0), UNSUP), (dict(N=1 << 20), UNSUP), (dict(N=1 << 30), UNSUP), (dict(K=1 << 21), UNSUP), (dict(dy=None), BAD),
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(z=None), BAD), (dict(z=None, act=0), BAD), (dict(dx=17), BAD), (dict(dw=17), BAD),
    (dict(db=17), BAD), (dict(x=17), BAD), (dict(z=17), BAD), (dict(dx=None, dw=None, db=None), gb.OK),
    (dict(M=0, dw=None, db=None, dy=None), gb.OK), (dict(N=0, dx=None, dy=None), gb.OK), (dict(K=0, db=None, dy=None), gb.OK),
])
def test_backward_refusals(kw, want):
    assert back(**kw) == want


def test_workspaces():
    lib, n, m = gb.load(), ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.gemm_bt_gated_workspace_size(4, 4, 4, gb.BF16, gb.BF16, None) == BAD
    assert lib.gemm_bt_gated_workspace_size(4, 1 << 30, 4, gb.BF16, gb.BF16, ctypes.byref(n)) == UNSUP
    assert lib.gemm_bt_gated_workspace_size(-1, 4, 4, gb.BF16, gb.BF16, ctypes.byref(n)) == BAD and n.value == 0
    for M, N, K in ((64, 4096, 8192), (512, 512, 16384), (4096, 4096, 4096)):
        assert lib.gemm_bt_gated_workspace_size(M, N, K, gb.BF16, gb.BF16, ctypes.byref(n)) == gb.OK
        assert lib.gemm_bt_epi_workspace_size(M, 2 * N, K, gb.BF16, gb.BF16, ctypes.byref(m)) == gb.OK and n.value == m.value
    f = lib.gemm_bt_gated_backward_workspace
    assert f(4, 4, 4, 0, None) == BAD and f(4, 4, 4, 5, ctypes.byref(n)) == BAD and f(4, 1 << 30, 4, 0, ctypes.byref(n)) == UNSUP
    assert f(100, 256, 64, 0, ctypes.byref(n)) == gb.OK and n.value >= 100 * 512 * 2  # dz for every activation
    assert f(0, 256, 64, 0, ctypes.byref(n)) == gb.OK and n.value == 0


def test_wrappers_check_before_the_library():
    x, w = torch.zeros(2, 16).bfloat16(), torch.zeros(4, 16).bfloat16()
    for call in (lambda: gb.gated_linear(x, w), lambda: gb.gated_linear_backward(x, x, w, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_wrapper_refusals(gpu):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    x, w, dy, pre = z(4, 16), z(8, 16), z(4, 4), z(4, 8)
    for error, call in ((ValueError, lambda: gpu.gated_linear(x, z(7, 16))), (ValueError, lambda: gpu.gated_linear(x, z(8, 15))),
                        (ValueError, lambda: gpu.gated_linear(x, w, bias=z(4))), (ValueError, lambda: gpu.gated_linear(x, w, activation="swish")),
                        (ValueError, lambda: gpu.gated_linear(x, w, out=z(4, 8))), (TypeError, lambda: gpu.gated_linear(x.float(), w.float())),
                        (TypeError, lambda: gpu.gated_linear(x, w.half())), (TypeError, lambda: gpu.gated_linear(x, w, out_dtype=torch.int8)),
                        (ValueError, lambda: gpu.gated_linear(x, w, x_scale=torch.ones(3, device="cuda"))),
                        (ValueError, lambda: gpu.gated_linear(x, w, weight_scale=torch.ones(4, device="cuda"))),
                        (ValueError, lambda: gpu.gated_linear_backward(dy, x, w, pre[:, :4])),
                        (ValueError, lambda: gpu.gated_linear_backward(pre, x, w, pre)),
                        (TypeError, lambda: gpu.gated_linear_backward(dy.float(), x, w, pre)),
                        (TypeError, lambda: gpu.gated_linear_backward(dy, x, w, pre.to(torch.int8)))):
        with pytest.raises(error):
            call()
