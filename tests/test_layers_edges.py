"""The row operators and the product with an epilogue at the edges of what they take: sizes of zero, operands in each
other's place, large extents, tails of the activations.  Tolerances stand beside the checks."""
import ctypes
import itertools
import math

import pytest

import dense_tiled_gemm_amd as gb

torch = pytest.importorskip("torch")

BAD, UNSUP = gb.ERR_INVALID_VALUE, gb.ERR_UNSUPPORTED
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
u = 2.0 ** -24


def say(*a):
    print("[case]", *a, flush=True)


def randn(seed, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def handle():
    return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------ rows of no elements

def test_rows_of_no_elements_need_a_place_for_their_scales():
    lib = gb.load()
    assert lib.gemm_bt_quantize_rows(None, 0, None, None, 3, 0, gb.BF16, gb.INT8, None) == BAD
    assert lib.gemm_bt_rms_norm(None, 0, None, 0, None, None, None, None, None, 3, 0, 1e-6, gb.BF16, gb.BF16, gb.INT8,
                                None) == BAD
    assert lib.gemm_bt_rms_norm(None, 0, None, 0, None, None, None, None, 18, 3, 0, 1e-6, gb.BF16, gb.BF16, gb.BF16,
                                None) == BAD


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 5, 3000])
def test_rows_of_no_elements(gpu, rows):
    """Their scales are the smallest there is and their rstd that of a mean of 0; a product with them is the empty sum."""
    lib = gpu.load()
    for eps, rstd_want in ((1e-6, 1e3), (0.25, 2.0), (0.0, float("inf"))):
        say("empty rows", rows, eps)
        scale, rstd = torch.full((rows + 1,), 7.0, device="cuda"), torch.full((rows + 1,), 7.0, device="cuda")
        assert lib.gemm_bt_rms_norm(None, 0, None, 0, None, None, None, scale.data_ptr(), rstd.data_ptr(), rows, 0, eps, gpu.BF16,
                                    gpu.BF16, gpu.INT8, handle()) == gpu.OK
        assert bool((scale[:rows] == 2.0 ** -100).all())
        # eps is rounded to fp32, then a root and a quotient: 3 u
        got = rstd[:rows].double()
        assert bool((got == rstd_want).all()) if math.isinf(rstd_want) else bool(((got - rstd_want).abs() <= 3 * u * rstd_want).all())
        assert float(scale[rows]) == 7.0 and float(rstd[rows]) == 7.0
        rstd.fill_(7.0)  # float rows: no scales, which are left as they are
        scale.fill_(7.0)
        assert lib.gemm_bt_rms_norm(None, 0, None, 0, None, None, None, scale.data_ptr(), rstd.data_ptr(), rows, 0, eps, gpu.F32,
                                    gpu.F32, gpu.F32, handle()) == gpu.OK
        assert bool((scale == 7.0).all()) and bool((rstd[:rows] != 7.0).all())
    scale = torch.full((rows,), float("nan"), device="cuda")
    assert lib.gemm_bt_quantize_rows(None, 0, None, scale.data_ptr(), rows, 0, gpu.F32, gpu.FP8_E4M3, handle()) == gpu.OK
    assert bool((scale == 2.0 ** -100).all())
    x, w = torch.empty(rows, 0, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.bfloat16, device="cuda")
    q = gpu.quantize_rows(x.view(1, rows, 0), torch.int8)
    assert q.q.shape == (1, rows, 0) and q.scale.shape == (1, rows) and bool((q.scale == 2.0 ** -100).all())
    n = gpu.add_rms_norm(x, w, residual=x, eps=0.25, out_dtype=torch.int8, save_rstd=True)
    assert n.h.shape == (rows, 0) and bool((n.scale == 2.0 ** -100).all()) and bool((n.rstd == 2.0).all())
    b = randn(1, 9).cuda()
    y = gpu.linear(n.y, torch.empty(9, 0, dtype=torch.int8, device="cuda"), bias=b, x_scale=n.scale, out_dtype=torch.float32)
    assert torch.equal(y, b.expand(rows, 9))
    dx, dw = gpu.add_rms_norm_backward(x, x, w, n.rstd)
    assert dx.shape == (rows, 0) and dw.shape == (0,)


# ------------------------------------------------------------------ operands in each other's place

@pytest.mark.parametrize("rows,d", [(2, 8), (256, 4096), (8192, 4096), (2, 100000)])
def test_norm_backward_not_in_place_of_h(rows, d):
    """dweight is summed from dy and h by other workgroups than those that write dx: neither may be overwritten."""
    f = gb.load().gemm_bt_rms_norm_backward
    call = lambda dx, dh: f(16, d, 32, d, 16, 16, dh, d, dx, 16, rows, d, gb.BF16, gb.BF16, 16, 1 << 40, None)
    for dh in (None, 48, 32):
        assert call(16, dh) == BAD and call(32, dh) == BAD


# ------------------------------------------------------------------ the workspace of split products

def split_operands(N=512, K=8192, seed=1):
    return (randn(seed, 8, K, std=3.0, dtype=torch.bfloat16).cuda(), randn(seed + 1, N, K, std=3.0, dtype=torch.bfloat16).cuda())


@pytest.mark.gpu
def test_workspace_is_cleared_in_the_order_of_its_stream(gpu):
    """A split product on an idle stream, called while torch's current stream is busy and memory holds other values."""
    a, b = randn(3, 512, 32768, dtype=torch.bfloat16).cuda(), randn(4, 1024, 32768, dtype=torch.bfloat16).cuda()
    assert gpu.gemm_bt_workspace_size(512, 1024, 32768, gpu.BF16, gpu.F32) > 0
    want = gpu.mm_bt(a, b, out_dtype=torch.float32)
    torch.cuda.synchronize()
    for _ in range(3):
        say("mm_bt on another stream")
        side = torch.cuda.Stream()
        gpu._ws_cache.pop((a.device.index, side.cuda_stream), None)
        out = torch.empty_like(want)
        left = [torch.full((20 << 20,), 0x5B, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del left  # what the next tensors are made of
        busy = torch.randn(2048, 2048, device="cuda")
        for _ in range(20):
            busy = busy @ busy * 0.01
        gpu.mm_bt(a, b, out_dtype=torch.float32, out=out, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(out, want)
        torch.cuda.synchronize()
        assert int(gpu.workspace_for(a.device, side.cuda_stream, 0)[:gpu.SK_COUNTER_BYTES].count_nonzero()) == 0


@pytest.mark.gpu
def test_workspace_of_a_captured_product_is_the_graphs(gpu):
    """Split products captured before and after eager ones on the same stream: neither shares the other's counters, and a
    larger workspace later on takes nothing from the graph."""
    x, w = split_operands()
    p, q = randn(5, 64, 8192, dtype=torch.bfloat16).cuda(), randn(6, 8192, 8192, dtype=torch.bfloat16).cuda()
    small = gpu.gemm_bt_plan_epi(8, 512, 8192, gpu.BF16, gpu.BF16)
    assert small.split_tiles > 0 and gpu.gemm_bt_workspace_size(64, 8192, 8192, gpu.BF16, gpu.BF16) > small.workspace_bytes
    wide = randn(7, 512, 32768, dtype=torch.bfloat16).cuda(), randn(8, 1024, 32768, dtype=torch.bfloat16).cuda()
    want, want_wide, want_q = gpu.linear(x, w), gpu.mm_bt(*wide), gpu.mm_bt(p, q)
    torch.cuda.synchronize()
    for first in (False, True):  # an eager product on the stream before the capture, or none
        say("captured mm_bt and linear", first)
        side = torch.cuda.Stream()
        gpu._ws_cache.pop((x.device.index, side.cuda_stream), None)
        if first:
            with torch.cuda.stream(side):
                gpu.linear(x, w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got_wide, got = gpu.mm_bt(*wide), gpu.linear(x, w)
        with torch.cuda.stream(side):
            assert torch.equal(gpu.linear(x, w), want)  # before the graph has run
            assert torch.equal(gpu.mm_bt(p, q), want_q)  # a larger workspace
        for _ in range(3):
            junk = torch.full((64 << 20,), 0x5B, dtype=torch.uint8, device="cuda")
            got.zero_(), got_wide.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want) and torch.equal(got_wide, want_wide)
            with torch.cuda.stream(side):
                assert torch.equal(gpu.linear(x, w), want)
            del junk


@pytest.mark.gpu
def test_products_on_a_stream_copy_their_operands_there(gpu):
    """mm_bt and mm on a stream whose operands are strided and still being written on it, while torch's current stream is idle."""
    a0, b0 = randn(1, 96, 512, dtype=torch.bfloat16), randn(2, 256, 512, dtype=torch.bfloat16)
    want = gpu.mm_bt(a0.cuda(), b0.cuda())
    want2 = gpu.mm(a0.cuda(), b0.t().contiguous().cuda())
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        say("mm_bt and mm of strided operands", type(stream).__name__)
        at, bt = torch.zeros(512, 96, dtype=torch.bfloat16, device="cuda"), torch.zeros(256, 1024, dtype=torch.bfloat16, device="cuda")
        src_a, src_b = a0.t().contiguous().cuda(), b0.cuda()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            busy = torch.randn(2048, 2048, device="cuda")
            for _ in range(20):
                busy = busy @ busy * 0.01
            at.copy_(src_a)
            bt[:, ::2].copy_(src_b)
        got = gpu.mm_bt(at.t(), bt[:, ::2], stream=stream)
        got2 = gpu.mm(at.t(), bt[:, ::2].t(), stream=stream)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(got2, want2)


# ------------------------------------------------------------------ wide results: the backward pass of a large vocabulary

def back_bytes(M, N, K, act=0):
    n = ctypes.c_size_t()
    assert gb.load().gemm_bt_linear_backward_workspace(M, N, K, act, ctypes.byref(n)) == gb.OK
    return n.value


def test_wide_linear_backward_is_not_cut_for_its_width():
    """dX = dz W reads dz row by row and W in steps of 64 rows: only a run of W past 2 GiB has to be cut, however wide dz
    is.  dW = dz^T X reads dz in steps of 64 rows and is cut past 2 GiB of it.  Without slices (these dX have tiles enough
    for every compute unit) the workspace holds the bias's partial sums alone, a few rows of them."""
    for M, N, K in ((8192, 128256, 4096), (4096, 151936, 4096), (8192, 40000, 4096), (4096, 256000, 2304)):
        assert M * N * 2 < 1 << 31
        assert back_bytes(M, N, K) < 64 * N * 4, (M, N, K)
    for M, N, K in ((16384, 128256, 4096), (8192, 151936, 4096)):  # dW in two slices, dX still whole
        assert 2 * N * K * 4 <= back_bytes(M, N, K) < 2 * N * K * 4 + 64 * N * 4, (M, N, K)
    M, N, K = 8192, 1 << 20, 2048  # W itself past 2 GiB: dX in slices too (and dW in 9)
    assert back_bytes(M, N, K) >= 2 * M * K * 4 + 9 * N * K * 4


@pytest.mark.gpu
def test_wide_linear_backward(gpu):
    """All of dX and dW of a wide result, in one run each, against 64 bits on the GPU: sums of N and M terms, N u and M u
    times the sum of magnitudes, then one rounding into bf16 (2^-8 relative, a little over half its last place)."""
    M, N, K = 4096, 33000, 4096
    say("linear backward", M, N, K)
    assert back_bytes(M, N, K) < 64 * N * 4
    g = torch.Generator(device="cuda").manual_seed(1)
    dy, x, w = ((torch.randn(*s, generator=g, device="cuda") * std).bfloat16() for s, std in (((M, N), 0.1), ((M, K), 1.0), ((N, K), 0.02)))
    got = gpu.linear_backward(dy, x, w)
    for name, g, (a, b), terms in (("dx", got.dx, (dy, w), N), ("dw", got.dweight, (dy.t(), x), M)):
        a, b = a.double().contiguous(), b.double()
        want = a @ b
        bound = 2.0 ** -8 * want.abs() + terms * u * (a.abs() @ b.abs())
        assert bool(((g.double() - want).abs() <= bound).all()), name
    want = dy.double().sum(0)
    assert bool(((got.dbias.double() - want).abs() <= 2.0 ** -8 * want.abs() + (M + 8) * u * dy.double().abs().sum(0)).all())


# ------------------------------------------------------------------ few rows

@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_few_rows_with_and_without_a_workspace(gpu, dt):
    """16-bit products of 16 rows and fewer whose plan needs no workspace: streamed without one, as the torch wrapper calls
    them, and on tiles with one.  The sum of K terms is within K u of the sum of their magnitudes, the bias adds u."""
    from dense_tiled_gemm_amd.layers import Epilogue

    lib, code = gpu.load(), {"bf16": gpu.BF16, "f16": gpu.F16}[dt]
    for M, N, K in ((16, 4096, 1024), (16, 4096, 1000), (16, 1024, 2048), (8, 2048, 1024), (1, 4096, 1536), (3, 1111, 1999), (16, 4096, 0)):
        say("few rows", M, N, K, dt)
        p = gpu.gemm_bt_plan_epi(M, N, K, code, gpu.F32)
        assert p.workspace_bytes == 0 and p.kernel != 3
        x, w, b = randn(1, M, K, dtype=DT[dt]), randn(2, N, K, dtype=DT[dt]), randn(3, N)
        want = x.double() @ w.double().t() + b.double()
        bound = (K + 1) * u * (x.double().abs() @ w.double().abs().t()) + 2 * u * want.abs()
        x, w, b = x.cuda(), w.cuda(), b.cuda()
        e = Epilogue(bias=b.data_ptr(), bias_dtype=gpu.F32)
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        got = [gpu.linear(x, w, bias=b, out_dtype=torch.float32)]
        for at, size in ((None, 0), (ws.data_ptr(), ws.numel())):
            got.append(torch.full((M, N), float("nan"), device="cuda"))
            assert lib.gemm_bt_epi(x.data_ptr(), w.data_ptr(), got[-1].data_ptr(), M, N, K, code, gpu.F32, ctypes.byref(e), at, size,
                                   handle()) == gpu.OK
        assert torch.equal(got[0], got[1])
        for c in got:
            assert bool(((c.cpu().double() - want).abs() <= bound).all())
        assert int(ws.count_nonzero()) == 0


# ------------------------------------------------------------------ 8-bit rows whose values leave fp32's range

@pytest.mark.gpu
@pytest.mark.parametrize("d", [2, 9, 600, 4096, 20000])
def test_rows_that_overflow_have_no_scale(gpu, d):
    """y = h rstd w past fp32's largest value is an infinity, and so the row's scale a NaN; the rows beside it, below that
    value, keep theirs: amax / Q within the norm's own (64 + d / 2048) u and 4 u for the scale's steps."""
    x = torch.zeros(4, d)
    x[0, 0], x[1, d - 1], x[3, 0], x[3, d // 2] = 1.0, -3.0, 1.0, 1.0
    w = torch.ones(d)
    # rstd is sqrt(d): the largest y is sqrt(d) w, 1.06 times the largest fp32 value in row 0 (w[0]); finite in row 1
    w[0], w[d - 1] = 1.06 * torch.finfo(torch.float32).max / math.sqrt(d), 0.9 * torch.finfo(torch.float32).max / math.sqrt(d)
    say("overflow", d)
    assert bool(torch.isinf(gpu.add_rms_norm(x.cuda(), w.cuda(), eps=0.0).y[0, 0]))
    for qt, q in ((torch.float8_e4m3fn, 448.0), (torch.int8, 127.0)):
        n = gpu.add_rms_norm(x.cuda(), w.cuda(), eps=0.0, out_dtype=qt)
        s = n.scale.cpu().double()
        assert math.isnan(s[0]) and math.isnan(s[2])  # (a row of zeros without eps: 0 / 0)
        for row in (1, 3):
            y = x[row].double() / x[row].double().square().mean().sqrt() * w.double()
            want = float(y.abs().max()) / q
            assert abs(float(s[row]) - want) <= (64 + d / 2048 + 4) * u * want, (row, d)


# ------------------------------------------------------------------ evenly spaced rows of more than two dimensions

def evenly_spaced():
    """(tensor on the CPU, whether its rows are evenly spaced and at least their length apart)."""
    t = randn(1, 4, 6, 96, dtype=torch.bfloat16)
    return [(t, True), (t[..., 32:64], True), (t[..., :1], True), (t[1:3, :, 5:50], True), (t[:, 2:3, 1:95], True), (t[0:1, :, :40], True),
            (t.view(2, 2, 6, 96)[..., 8:], True), (t[:, ::2], True), (t[::2, 0], True), (t[0, 0, 3:90], True), (t[:, :5], False),
            (t[::2, ::2, :8], False), (t.view(2, 2, 6, 96)[:, :1, :, :9], False), (t.transpose(0, 1), False), (t.transpose(1, 2), False), (t[..., ::2], False), (t[:, :1].expand(4, 6, 96), False),
            (t[:1].expand(4, 6, 96), False), (t[:, 0, None].expand(4, 3, 96), False), (t.as_strided((3, 5, 8), (40, 8, 1)), True),
            (t.as_strided((3, 5, 8), (20, 4, 1)), False), (t.as_strided((3, 5, 8), (60, 12, 1)), True)]


@pytest.mark.parametrize("i", range(len(evenly_spaced())))
def test_evenly_spaced_rows_are_not_copied(i):
    from dense_tiled_gemm_amd.layers import _rows

    t, even = evenly_spaced()[i]
    got, ld, rows, d = _rows(t, "t")
    assert (rows, d) == (math.prod(t.shape[:-1]), t.shape[-1])
    assert torch.equal(got.as_strided((rows, d), (ld, 1)), t.reshape(rows, d)) and ld >= d
    assert (got is t) == even


@pytest.mark.gpu
def test_norm_of_evenly_spaced_rows(gpu):
    """Norm, quantisation and gradient of slices of three and four dimensions: the bits of their contiguous copies."""
    for i, (t, _) in enumerate(evenly_spaced()):
        say("rows of", tuple(t.shape), t.stride())
        base = torch.zeros(4 * 6 * 96, dtype=t.dtype, device="cuda")
        base.copy_(torch.as_strided(t, (base.numel(),), (1,), 0))
        x = base.as_strided(t.shape, t.stride(), t.storage_offset())
        c = x.contiguous()
        w = (1 + randn(2, t.shape[-1], std=0.2)).cuda()
        a, b = (gpu.add_rms_norm(v, w, residual=v, out_dtype=torch.float32, save_rstd=True) for v in (x, c))
        assert a.y.shape == t.shape and torch.equal(a.y, b.y) and torch.equal(a.h, b.h) and torch.equal(a.rstd, b.rstd)
        a, b = gpu.quantize_rows(x, torch.int8), gpu.quantize_rows(c, torch.int8)
        assert torch.equal(a.q, b.q) and torch.equal(a.scale, b.scale)
        rstd = torch.ones(t.shape[:-1], device="cuda")
        a, b = (gpu.add_rms_norm_backward(v, v, w, rstd, dh=v) for v in (x, c))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(base.cpu(), torch.as_strided(t, (base.numel(),), (1,), 0))


# ------------------------------------------------------------------ 8-bit operands off a 16-byte boundary

@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.int8, torch.float8_e4m3fn, torch.float8_e5m2])
def test_linear_of_eight_bits_from_any_start(gpu, dt):
    """x and the weight as views that start off a 16-byte boundary: the bits of the aligned ones."""
    for M, N, K in ((3, 40, 64), (16, 8192, 512), (100, 300, 1024), (64, 512, 8192)):
        x, w = randn(1, M, K, std=3.0).to(dt).cuda(), randn(2, N, K, std=3.0).to(dt).cuda()
        b = randn(3, N).cuda()
        want = gpu.linear(x, w, bias=b, activation="relu")
        for off_x, off_w in ((1, 0), (0, 8), (5, 15)):
            say("eight bits", M, N, K, dt, off_x, off_w)
            moved = []
            for t, off in ((x, off_x), (w, off_w)):
                buf = torch.zeros(t.numel() + 16, dtype=torch.uint8, device="cuda").view(dt)
                v = buf[off:off + t.numel()].view(t.shape)
                v.copy_(t)
                assert v.data_ptr() % 16 == off
                moved.append(v)
            assert torch.equal(gpu.linear(*moved, bias=b, activation="relu"), want)


# ------------------------------------------------------------------ refusals of the wrappers

@pytest.mark.gpu
def test_h_out_needs_a_residual(gpu):
    x, w = randn(1, 3, 16).cuda(), torch.ones(16, device="cuda")
    h = torch.full_like(x, 7.0)
    with pytest.raises(ValueError, match="residual"):
        gpu.add_rms_norm(x, w, h_out=h)
    assert bool((h == 7.0).all())
    assert gpu.add_rms_norm(x, w, residual=x, h_out=h).h is h and torch.equal(h, x + x)


# ------------------------------------------------------------------ tails of the activations

def tail_points():
    """Zeros, both signs, steps of 1/16 in the middle and the largest arguments whose results are normal fp32 numbers."""
    z = torch.cat([torch.linspace(-87, 87, 2785), torch.linspace(-13, 13, 6657), randn(1, 2000, std=3.0), randn(2, 200, std=1e-3)])
    return z.float()


def act_and_units(z, act):
    """act(z) in 64 bits, its derivative, and the relative error the header allows in units of 2^-24."""
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p), 8 + 1.5 * z.abs()
    if act == "gelu":
        # ndtr below -5 from the asymptotic continued fraction of Mills' ratio, whose error there is below 1e-12
        x = z.abs().clamp_min(5.0)
        f = x
        for k in range(60, 0, -1):
            f = x + k / f
        density = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        phi = torch.where(z < -5, density / f, torch.special.ndtr(z))
        return z * phi, phi + z * density, 24 + 1.25 * z * z
    a = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(a)
    return z * p, p + z * p * (1 - p) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z), 8 + 6 * a.abs()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_tails_of_the_activations(gpu, act):
    """fp32 results, relative to themselves.  The units: the exponential's argument carries one rounding of z (silu), two of
    z z / 2 or five of gelu_tanh's cubic, times log2(e) rounded twice more, each as large as the argument; the exponential,
    the reciprocal, the sum and the product are 8 more at most; Phi's polynomial of t = 1 / (1 + |z| / 4) 16 more (t's 3 by
    the polynomial's condition of 3.2, its steps 3.4, its fit 0.8).  Below 2^-126 |z| a result may be 0."""
    z = tail_points()
    want, slope, units = act_and_units(z.double(), act)
    bound = units * u * want.abs() + 2.0 ** -125 * z.double().abs()
    assert bool((want[z < -4].abs() > 4 * bound[z < -4])[z[z < -4] > (-80 if act == "silu" else -6)].all())  # 0 would not pass
    n, gz = z.numel(), z.cuda()
    for M, K in ((1, 0), (3, 64), (300, 64)):  # the empty sum, the streaming kernel, tiles
        say("tails", act, M, K)
        x, w = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), torch.ones(n, K, dtype=torch.bfloat16, device="cuda")
        y = gpu.linear(x, w, bias=gz, activation=act, out_dtype=torch.float32).cpu().double()
        bad = ((y - want).abs() > bound).any(0)
        assert not bool(bad.any()), (act, z[bad][:5], y[0, bad][:5], want[bad][:5])
    dz, dy = torch.empty(1, n, device="cuda"), torch.ones(1, n, device="cuda")
    assert gpu.load().gemm_bt_act_backward(dy.data_ptr(), gz.data_ptr(), dz.data_ptr(), None, 1, n, {"silu": 4, "gelu": 2, "gelu_tanh": 3}[act],
                                           gpu.F32, gpu.F32, gpu.F32, None, 0, handle()) == gpu.OK
    off = (dz[0].cpu().double() - slope).abs() - (2.0 ** -19 * (1 + z.double().abs()))
    assert bool((off <= 0).all()), (act, z[off > 0][:5])


# ------------------------------------------------------------------ results in an input's place, rows of odd length

@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(5, 9), (700, 63), (1200, 513), (3, 1031), (700, 1031), (600, 4097), (300, 16383), (3, 20001)])
def test_odd_rows_in_place(gpu, rows, d):
    """The last load of a row of odd length begins inside the chunk before, which another thread may already have replaced:
    what it holds of that chunk is not used.  The bits are those of results of their own."""
    lib = gpu.load()
    x, r, dy = (randn(i, rows, d, dtype=torch.bfloat16).cuda() for i in range(3))
    w = (1 + randn(4, d, std=0.3)).bfloat16().cuda()
    want = gpu.add_rms_norm(x, w, residual=r, save_rstd=True)
    for into in (0, 1):
        say("odd rows in place", rows, d, into)
        pair = [x.clone(), r.clone()]
        got = gpu.add_rms_norm(pair[0], w, residual=pair[1], h_out=pair[into], save_rstd=True)
        assert torch.equal(pair[into], want.h) and torch.equal(got.y, want.y) and torch.equal(got.rstd, want.rstd)
    dx, dw = gpu.add_rms_norm_backward(dy, want.h, w, want.rstd, dh=r)
    need = ctypes.c_size_t()
    assert lib.gemm_bt_rms_norm_backward_workspace(rows, d, ctypes.byref(need)) == gpu.OK
    ws, dh, dw2 = torch.empty(need.value + 16, dtype=torch.uint8, device="cuda"), r.clone(), torch.empty_like(dw)
    assert lib.gemm_bt_rms_norm_backward(dy.data_ptr(), d, want.h.data_ptr(), d, w.data_ptr(), want.rstd.data_ptr(), dh.data_ptr(), d,
                                         dh.data_ptr(), dw2.data_ptr(), rows, d, gpu.BF16, gpu.BF16, ws.data_ptr(), need.value,
                                         handle()) == gpu.OK
    assert torch.equal(dh, dx) and torch.equal(dw2, dw)
    dz, place = torch.empty_like(dy), dy.clone()
    for out, src in ((dz, dy), (place, place)):
        assert lib.gemm_bt_act_backward(src.data_ptr(), x.data_ptr(), out.data_ptr(), None, rows, d, 4, gpu.BF16, gpu.BF16, gpu.BF16, None, 0,
                                        handle()) == gpu.OK
    assert torch.equal(dz, place)
