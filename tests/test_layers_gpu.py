"""The row operators and the product with an epilogue on the GPU, against plain implementations in 64 bits on the CPU.

Where the tolerances come from (u = 2^-24, the unit roundoff of fp32; U that of the stored type):
  * a norm's row: h is one rounding of x + residual; the sum of squares passes at most 16 + 6 + 16 additions in a
    register, over a wave and over a workgroup (rows of up to 16384; longer ones 8 more per 8192 elements), so rstd is
    within (60 + d/2048) u and y = h * rstd * w three roundings more: Y_REL(d) = (64 + d/2048) u; then one rounding into
    the stored type, U |y|, or half its smallest step near zero;
  * a product's sum of K terms: K u sum |a b| (any order of fp32 additions);
  * an activation: its exponential's argument carries |z| 2^-23, which moves a sigmoid by p (1 - p) |z| 2^-23 < 2^-24
    and, with the exponential's and the reciprocal's own errors, by at most 2^-21 in all; Phi likewise (its polynomial
    is within 2^-21 of it): ACT = 2^-20 |z|.  None of the activations is steeper than 1.13;
  * a slope: the same for its first term; the second is z times a product of such factors: 2^-20 (1 + |z|^3);
  * sums over M rows: M u sum |terms|.
"""
import itertools
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EIGHT = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
QMAX = {"e4m3": 448.0, "i8": 127.0}
u = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: u}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}  # half a step, or above it
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def say(*a):
    print("[case]", *a, flush=True)


def y_rel(d):
    return (64 + d / 2048) * u


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(seed, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen(seed)) * std).to(dtype)


def close(got, want, tol, what):
    """|got - want| <= tol + the rounding of got's type, entry for entry; NaN and infinities where they are wanted."""
    got = got.detach().cpu()
    bound = tol + UNIT[got.dtype] * want.abs() * (1 + 1e-6) + TINY[got.dtype]
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    bad = fine & ((got - want).abs() > bound)
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError((what, int(bad.sum()), at, float(got[at]), float(want[at]), float(bound.expand_as(want)[at])))


def guarded(shape, dtype, offset=0, guard=256):
    """A tensor inside a larger buffer, `offset` elements past 16-byte alignment, and a check that nothing around it changed."""
    n = math.prod(shape)
    size = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full(((n + 2 * guard + offset + 16) * size,), 0x5B, dtype=torch.uint8, device="cuda")
    at = guard + offset
    t = raw.view(dtype)[at:at + n].view(shape)

    def untouched():
        torch.cuda.synchronize()
        assert bool((raw[:at * size] == 0x5B).all()) and bool((raw[(at + n) * size:] == 0x5B).all()), "wrote outside"
    return t, untouched


# ------------------------------------------------------------------ norm and 8-bit rows

def norm64(x, r, w, eps):
    h = x.double() + (0 if r is None else r.double())
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return h, rstd, h * rstd * w.double()


def code_values(q):
    return q.float().double().cpu()


def check_codes(q, scale, y64, qt, rel, what):
    """q and its scales against the exact rows y64, known to a relative error `rel`."""
    amax = y64.abs().amax(-1)
    want = torch.clamp(amax / QMAX[qt], min=2.0 ** -100)
    s = scale.cpu().double()
    assert bool(((s - want).abs() <= (rel + 4 * u) * want).all()), what
    v = y64 / want[..., None]
    got = code_values(q)
    if qt == "i8":
        half = torch.full_like(v, 0.5)
    else:  # half a step of E4M3: 3 bits after the leading one, smallest exponent -6
        half = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 4)
        # a value just below a power of two may round as the one above it does
        half = torch.maximum(half, torch.exp2(torch.floor(torch.log2((v.abs() * (1 + 1e-5)).clamp_min(2.0 ** -6))) - 4))
    assert bool(((got - v).abs() <= half + (2 * rel + 16 * u) * v.abs()).all()), what
    assert bool((got.abs() <= QMAX[qt]).all()), what
    top = amax > 2.0 ** -90  # the largest magnitude of a row takes the largest code
    assert bool((got.abs().amax(-1)[top] == QMAX[qt]).all()), what


WIDTHS = [1, 2, 7, 8, 9, 63, 64, 130, 512, 513, 1000, 1024, 1031, 2048, 2049, 2056, 4096, 4097, 5000, 8192, 8200, 16384]


@pytest.mark.parametrize("d", WIDTHS)
def test_norm(gpu, d):
    rows_of = (1, 3, 5) if d > 600 else (1, 7, 1200)
    for rows, dt, out, wt, res in itertools.product(rows_of, ("bf16", "f16", "f32"), ("own", "e4m3", "i8"), ("own", "f32"), (0, 1)):
        if (rows + d + len(out) + res) % 2 and d > 9:  # half of the combinations at each width
            continue
        seed = 1000 * d + rows
        x = randn(seed, rows, d, std=2.0, dtype=DT[dt])
        r = randn(seed + 1, rows, d, std=3.0, dtype=DT[dt]) if res else None
        w = (1 + randn(seed + 2, d, std=0.3)).to(DT[dt] if wt == "own" else torch.float32)
        say("norm", rows, d, dt, out, wt, res, "seed", seed)
        y, untouched = guarded((rows, d), EIGHT.get(out, DT[dt]), offset=seed % 3)
        got = gpu.add_rms_norm(x.cuda(), w.cuda(), residual=None if r is None else r.cuda(), eps=1e-5,
                               out_dtype=y.dtype, save_rstd=True, out=y)
        untouched()
        h64, rstd64, y64 = norm64(x, r, w, 1e-5)
        close(got.rstd, rstd64[:, 0], y_rel(d) * rstd64[:, 0], "rstd")
        if res:
            close(got.h, h64, 2 * u * h64.abs(), "h")
        else:
            assert got.h is None
        if out == "own":
            assert got.scale is None
            close(got.y, y64, y_rel(d) * y64.abs(), "y")
        else:
            check_codes(got.y, got.scale, y64, out, y_rel(d), (rows, d, dt, out))


@pytest.mark.parametrize("rows,d", [(515, 4096), (513, 8192), (600, 3000), (700, 1500), (520, 12000), (2100, 700), (1300, 257),
                                    (2, 16392), (3, 33001), (1, 100003)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_many_and_long_rows(gpu, rows, d, dt):
    # more rows than two per CU take the other forms of the kernel; rows past 16384 are read once per statistic
    for out, res in (("own", 1), ("e4m3", 1), ("i8", 0)):
        seed = rows + d
        say("norm", rows, d, dt, out, res, "seed", seed)
        x, w = randn(seed, rows, d, dtype=DT[dt]), (1 + randn(seed + 2, d, std=0.3)).to(DT[dt])
        r = randn(seed + 1, rows, d, dtype=DT[dt]) if res else None
        got = gpu.add_rms_norm(x.cuda(), w.cuda(), residual=None if r is None else r.cuda(), out_dtype=EIGHT.get(out))
        h64, _, y64 = norm64(x, r, w, 1e-6)
        if res:
            close(got.h, h64, 2 * u * h64.abs(), "h")
        if out == "own":
            close(got.y, y64, y_rel(d) * y64.abs(), "y")
        else:
            check_codes(got.y, got.scale, y64, out, y_rel(d), (rows, d, dt, out))


def test_norm_layouts_and_places(gpu):
    # rows of a wider matrix, unaligned starts, three dimensions, every other row; h into x or into the residual itself
    wide = randn(5, 40, 700, dtype=torch.bfloat16).cuda()
    w = (1 + randn(6, 333, std=0.2)).cuda()
    for x in (wide[:, 3:336], wide[::2, 64:397], wide[1:, :333], wide.t()[:333].t()[:, :333]):
        r = wide[:x.shape[0], 350:683]
        _, _, y64 = norm64(x.cpu(), r.cpu(), w.cpu(), 1e-6)
        close(gpu.add_rms_norm(x, w, residual=r).y, y64, y_rel(333) * y64.abs(), "strided")
    cube = randn(7, 4, 5, 96, dtype=torch.float16).cuda()
    for x in (cube, cube.transpose(0, 1)):
        w96 = torch.ones(96, dtype=torch.float16, device="cuda")
        got = gpu.add_rms_norm(x, w96, residual=x, out_dtype=torch.float32, save_rstd=True)
        h64, rstd64, y64 = norm64(x.cpu(), x.cpu(), w96.cpu(), 1e-6)
        assert got.y.shape == x.shape and got.rstd.shape == x.shape[:-1]
        close(got.y, y64, y_rel(96) * y64.abs(), "cube")
        close(got.h, h64, 2 * u * h64.abs(), "cube h")
    for d, out in itertools.product((64, 4096, 20000), (None, torch.float8_e4m3fn)):
        x, r, w = randn(8, 6, d, dtype=torch.bfloat16), randn(9, 6, d, dtype=torch.bfloat16), torch.ones(d, dtype=torch.bfloat16)
        h64, _, y64 = norm64(x, r, w, 1e-6)
        for into in (0, 1):
            pair = [x.cuda(), r.cuda()]
            got = gpu.add_rms_norm(pair[0], w.cuda(), residual=pair[1], out_dtype=out, h_out=pair[into])
            assert got.h.data_ptr() == pair[into].data_ptr()
            close(pair[into], h64, 2 * u * h64.abs(), ("in place", d))
            assert torch.equal(pair[1 - into].cpu(), (x, r)[1 - into])
            if out is None:
                close(got.y, y64, y_rel(d) * y64.abs(), ("in place y", d))
            else:
                check_codes(got.y, got.scale, y64, "e4m3", y_rel(d), ("in place", d))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [40, 2048, 20000])
def test_norm_extremes(gpu, d, dt):
    """Rows of zeros, of the type's smallest and largest values, and rows with an infinity or a NaN: each row by itself."""
    big = torch.finfo(DT[dt]).max
    x = randn(3, 8, d)
    x[0] = 0.0
    x[1] = 2.0 ** -20
    x[2, :] = 0.0
    x[2, d - 1] = 3.0
    x[3, d // 2] = float("inf")
    x[4, d - 1] = float("nan")
    x[5, 0] = -float("inf")
    x[6] = 1e18 if dt != "f16" else big / 2
    x = x.to(DT[dt])
    w = torch.ones(d)
    say("norm extremes", d, dt)
    got = gpu.add_rms_norm(x.cuda(), w.cuda(), eps=1e-6, save_rstd=True)
    y = got.y.cpu().double()
    _, _, y64 = norm64(x, None, w, 1e-6)
    for row in (0, 1, 2, 6, 7):
        close(got.y[row], y64[row], y_rel(d) * y64[row].abs(), (row, d, dt))
    for row in (3, 5):  # rstd = 0: zeros, and infinity * 0
        keep = torch.isfinite(x[row])
        assert bool((y[row][keep] == 0).all()) and bool(torch.isnan(y[row][~keep]).all())
    assert bool(torch.isnan(y[4]).all())
    for qt in ("e4m3", "i8"):
        q = gpu.quantize_rows(x.cuda(), EIGHT[qt])
        s = q.scale.cpu()
        assert bool(torch.isnan(s[[3, 4, 5]]).all())
        rows = [0, 1, 2, 6, 7]
        check_codes(q.q[rows], q.scale[rows], x[rows].double(), qt, 0.0, ("quantize", d, dt))
        assert float(s[0]) == 2.0 ** -100 and bool((code_values(q.q[0]) == 0).all())
        n = gpu.add_rms_norm(x.cuda(), w.cuda(), out_dtype=EIGHT[qt])
        assert bool(torch.isnan(n.scale[[3, 4, 5]]).all()) and bool(torch.isfinite(n.scale[rows]).all())


def test_quantize_rows(gpu):
    for rows, d, dt, qt in itertools.product((0, 1, 5, 700), (1, 16, 48, 1000, 8192, 17000), ("bf16", "f16", "f32"), ("e4m3", "i8")):
        if rows == 700 and d > 1000:
            continue
        x = randn(rows + d, rows, d, std=4.0, dtype=DT[dt])
        say("quantize", rows, d, dt, qt)
        got = gpu.quantize_rows(x.cuda(), EIGHT[qt])
        assert got.q.shape == x.shape and got.scale.shape == (rows,)
        check_codes(got.q, got.scale, x.double(), qt, 0.0, (rows, d, dt, qt)) if rows else None
    # values that are exact in 8 bits come back as they are; ties go to the even code
    v = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 3.0]])
    assert gpu.quantize_rows(v.cuda(), torch.int8).q.cpu().tolist() == [[127, 0, 2, 2, 0, -2, -126, 3]]
    v = torch.tensor([[448.0, 1.0625, 1.1875, 17.0, -19.0, 2.0 ** -10, 3 * 2.0 ** -10, 416.0]])
    assert gpu.quantize_rows(v.cuda()).q.cpu().float().tolist() == [[448.0, 1.0, 1.25, 16.0, -20.0, 0.0, 2.0 ** -8, 416.0]]


# ------------------------------------------------------------------ norm, backward

def norm_back64(dy, h, w, rstd, dh):
    dy, h, w, rstd = dy.double(), h.double(), w.double(), rstd.double()[..., None]
    xhat, g = h * rstd, dy * w
    c = (g * xhat).mean(-1, keepdim=True)
    spread = (g * xhat).abs().mean(-1, keepdim=True)
    d = dy.shape[-1]
    dx = rstd * (g - xhat * c) + (0 if dh is None else dh.double())
    # each factor is a few roundings, the mean (64 + d/2048) more relative to the sum of magnitudes
    tol_dx = rstd * (8 * u * g.abs() + (y_rel(d) + 8 * u) * xhat.abs() * spread) + 2 * u * dx.abs()
    dw = (dy * xhat).flatten(0, -2).sum(0)
    rows = dy.flatten(0, -2).shape[0]
    tol_dw = (rows + 8) * u * (dy * xhat).abs().flatten(0, -2).sum(0)
    return dx, tol_dx, dw, tol_dw


@pytest.mark.parametrize("d", [1, 7, 8, 64, 100, 512, 520, 1000, 1031, 2048, 2050, 4096, 4099, 8192, 8200, 16384, 17001])
def test_norm_backward(gpu, d):
    for rows, dt, wt, res in itertools.product((1, 5, 300) if d <= 4096 else (1, 5), ("bf16", "f16", "f32"), ("own", "f32"), (0, 1)):
        seed = d + rows
        if (rows + d + res + len(wt)) % 2 and d > 8:
            continue
        h, dy = randn(seed, rows, d, std=2.0, dtype=DT[dt]), randn(seed + 1, rows, d, std=0.1, dtype=DT[dt])
        dh = randn(seed + 2, rows, d, std=0.1, dtype=DT[dt]) if res else None
        w = (1 + randn(seed + 3, d, std=0.3)).to(DT[dt] if wt == "own" else torch.float32)
        rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
        say("norm backward", rows, d, dt, wt, res, "seed", seed)
        got = gpu.add_rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dh=None if dh is None else dh.cuda())
        dx, tol_dx, dw, tol_dw = norm_back64(dy, h, w, rstd, dh)
        close(got[0], dx, tol_dx, ("dx", rows, d, dt))
        close(got[1], dw, tol_dw, ("dw", rows, d, dt))
        assert got[0].dtype == DT[dt] and got[1].dtype == w.dtype


@pytest.mark.parametrize("rows,d", [(3000, 200), (2500, 768), (1500, 2000), (1200, 4000), (700, 8000), (530, 10000)])
def test_norm_backward_many_rows(gpu, rows, d):
    # more rows than workgroups: each sums several rows
    for dt in ("bf16", "f32"):
        h, dy, dh = (randn(rows + i, rows, d, std=s, dtype=DT[dt]) for i, s in ((0, 2.0), (1, 0.1), (2, 0.1)))
        w = (1 + randn(3, d, std=0.3)).to(DT[dt])
        rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
        say("norm backward", rows, d, dt)
        args = [t.cuda() for t in (dy, h, w, rstd)]
        got = gpu.add_rms_norm_backward(*args, dh=dh.cuda())
        again = gpu.add_rms_norm_backward(*args, dh=dh.cuda())
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])  # the same bits on every run
        dx, tol_dx, dw, tol_dw = norm_back64(dy, h, w, rstd, dh)
        close(got[0], dx, tol_dx, ("dx", rows, d, dt))
        close(got[1], dw, tol_dw, ("dw", rows, d, dt))


@pytest.mark.parametrize("rows,d", [(1300, 505), (1300, 506), (1100, 1021), (600, 2042), (530, 4099), (520, 8188), (513, 9999),
                                    (3, 13), (70, 1022), (9, 9007), (1900, 1321), (2000, 2050)])
def test_ragged_rows(gpu, rows, d):
    """Rows that end inside a chunk, wider apart than they are long and with NaN between them, dx in place of dh."""
    import ctypes

    lib, need = gpu.load(), ctypes.c_size_t()
    codes = {torch.float32: gpu.F32, torch.float16: gpu.F16, torch.bfloat16: gpu.BF16}
    for dt, wt in (("bf16", "own"), ("f16", "f32"), ("f32", "own")):
        say("ragged rows", rows, d, dt, wt)
        wide = [torch.full((rows, d + 3 + i), math.nan, dtype=DT[dt]) for i in range(4)]
        x, r, dy, dh = (w[:, 1 + i % 3:1 + i % 3 + d] for i, w in enumerate(wide))
        for i, (t, std) in enumerate(((x, 2.0), (r, 1.0), (dy, 0.1), (dh, 0.1))):
            t.copy_(randn(d + i, rows, d, std=std, dtype=DT[dt]))
        w = (1 + randn(d + 4, d, std=0.3)).to(DT[dt] if wt == "own" else torch.float32)
        gx, gr, gdy, gdh = (wide[i].cuda()[:, 1 + i % 3:1 + i % 3 + d] for i in range(4))
        got = gpu.add_rms_norm(gx, w.cuda(), residual=gr, eps=1e-5, save_rstd=True)
        h64, rstd64, y64 = norm64(x, r, w, 1e-5)
        close(got.h, h64, 2 * u * h64.abs(), "h")
        close(got.rstd, rstd64[:, 0], y_rel(d) * rstd64[:, 0], "rstd")
        close(got.y, y64, y_rel(d) * y64.abs(), "y")
        q = gpu.quantize_rows(gx, torch.int8)
        check_codes(q[0], q[1], x.double(), "i8", y_rel(d), (rows, d, dt))
        h, rstd = got.h.cpu(), got.rstd.cpu()
        dx, dw = gpu.add_rms_norm_backward(gdy, got.h, w.cuda(), got.rstd, dh=gdh)
        want, tol_dx, want_dw, tol_dw = norm_back64(dy, h, w, rstd, dh)
        close(dx, want, tol_dx, ("dx", rows, d, dt))
        close(dw, want_dw, tol_dw, ("dw", rows, d, dt))
        there, gw, again = gdh.contiguous(), w.cuda(), torch.empty(d, dtype=w.dtype, device="cuda")
        assert lib.gemm_bt_rms_norm_backward_workspace(rows, d, ctypes.byref(need)) == gpu.OK
        ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
        assert lib.gemm_bt_rms_norm_backward(gdy.data_ptr(), gdy.stride(0), got.h.data_ptr(), d, gw.data_ptr(), got.rstd.data_ptr(),
                                             there.data_ptr(), d, there.data_ptr(), again.data_ptr(), rows, d, codes[DT[dt]],
                                             codes[w.dtype], ws.data_ptr(), need.value,
                                             torch.cuda.current_stream().cuda_stream) == gpu.OK
        assert torch.equal(there, dx) and torch.equal(again, dw)


@pytest.mark.parametrize("rows,n", [(5000, 60), (3000, 121), (2500, 250), (2100, 1022), (1700, 2051), (1100, 4097)])
def test_act_backward_ragged_many_rows(gpu, rows, n):
    """More rows than the lanes of a launch, so that each lane goes on through its rows."""
    import ctypes

    lib = gpu.load()
    for code, dt in ((gpu.BF16, "bf16"), (gpu.F32, "f32")):
        say("act backward ragged", rows, n, dt)
        dy, z = randn(n, rows, n, dtype=DT[dt]), randn(n + 1, rows, n, std=2.5, dtype=DT[dt])
        need = ctypes.c_size_t()
        assert lib.gemm_bt_act_backward_workspace(rows, n, ctypes.byref(need)) == gpu.OK
        ws, ws_ok = guarded((need.value,), torch.uint8)
        dz, dz_ok = guarded((rows, n), DT[dt], offset=n % 3)
        db, db_ok = guarded((n,), torch.float32)
        gdy, gz = dy.cuda(), z.cuda()
        assert lib.gemm_bt_act_backward(gdy.data_ptr(), gz.data_ptr(), dz.data_ptr(), db.data_ptr(), rows, n, ACTS.index("silu"),
                                        code, code, gpu.F32, ws.data_ptr(), need.value,
                                        torch.cuda.current_stream().cuda_stream) == gpu.OK
        for ok in (ws_ok, dz_ok, db_ok):
            ok()
        z64, dy64 = z.double(), dy.double()
        slope = slope64(z64, "silu")
        tol = dy64.abs() * 2.0 ** -20 * (1 + z64.abs() ** 3) + u * (dy64 * slope).abs()
        close(dz, dy64 * slope, tol, ("dz", rows, n, dt))
        close(db, (dy64 * slope).sum(0), tol.sum(0) + (rows + 4) * u * (dy64 * slope).abs().sum(0), ("db", rows, n, dt))


def test_norm_gradient_against_differences(gpu):
    """dx, dresidual and dw of L = sum(y * dy) + sum(h * dh) against central differences of the 64-bit forward pass."""
    rows, d = 3, 37
    x, r, dy, dh = (randn(20 + i, rows, d).double() for i in range(4))
    w = 1 + randn(30, d, std=0.3).double()

    def loss(x, r, w):
        h, _, y = norm64(x, r, w, 1e-3)
        return (y * dy).sum() + (h * dh).sum()

    f = gpu.add_rms_norm(x.float().cuda(), w.float().cuda(), residual=r.float().cuda(), eps=1e-3, save_rstd=True)
    dx, dw = gpu.add_rms_norm_backward(dy.float().cuda(), f.h, w.float().cuda(), f.rstd, dh=dh.float().cuda())
    step = 1e-5
    for i, j in ((0, 0), (1, 17), (2, 36)):
        for t in (x, r):
            e = torch.zeros_like(t)
            e[i, j] = step
            want = (loss(x + e, r, w) - loss(x - e, r, w)) / (2 * step)
            assert abs(float(dx[i, j]) - float(want)) <= 1e-5 * (1 + abs(float(want)))
        e = torch.zeros_like(w)
        e[j] = step
        want = (loss(x, r, w + e) - loss(x, r, w - e)) / (2 * step)
        assert abs(float(dw[j]) - float(want)) <= 1e-5 * (1 + abs(float(want)))


@pytest.mark.parametrize("rows,d", [(300, 512), (4000, 512), (2, 20000)])
def test_norm_backward_into_dh(gpu, rows, d):
    """dx may take the place of dh; not of dy, which the weight's gradient still reads."""
    import ctypes

    lib = gpu.load()
    dy, h, dh = (randn(i, rows, d, dtype=torch.bfloat16).cuda() for i in range(3))
    w, rstd = randn(3, d, dtype=torch.bfloat16).cuda(), (randn(4, rows).abs() + 0.5).cuda()
    want = gpu.add_rms_norm_backward(dy, h, w, rstd, dh=dh)
    need = ctypes.c_size_t()
    assert lib.gemm_bt_rms_norm_backward_workspace(rows, d, ctypes.byref(need)) == gpu.OK
    ws = torch.empty(max(need.value, 16), dtype=torch.uint8, device="cuda")
    dw = torch.empty_like(w)

    def call(dx, nbytes):
        return lib.gemm_bt_rms_norm_backward(dy.data_ptr(), d, h.data_ptr(), d, w.data_ptr(), rstd.data_ptr(), dh.data_ptr(), d,
                                             dx.data_ptr(), dw.data_ptr(), rows, d, gpu.BF16, gpu.BF16, ws.data_ptr(), nbytes,
                                             torch.cuda.current_stream().cuda_stream)
    assert call(dy, need.value) == gpu.ERR_INVALID_VALUE
    if need.value:
        assert call(dh, need.value - 4) == gpu.ERR_INVALID_VALUE
    assert call(dh, need.value) == gpu.OK
    assert torch.equal(dh, want[0]) and torch.equal(dw, want[1])


def test_norm_backward_layouts_and_no_rows(gpu):
    wide = randn(40, 30, 400, dtype=torch.bfloat16)
    dy, h, dh = wide[:, 1:130], wide[:, 130:259], wide[:, 260:389]
    w, rstd = randn(41, 129, dtype=torch.bfloat16), randn(42, 30).abs() + 0.5
    g = wide.cuda()
    got = gpu.add_rms_norm_backward(g[:, 1:130], g[:, 130:259], w.cuda(), rstd.cuda(), dh=g[:, 260:389])
    dx, tol_dx, dw, tol_dw = norm_back64(dy, h, w, rstd, dh)
    close(got[0], dx, tol_dx, "dx")
    close(got[1], dw, tol_dw, "dw")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dx, dw = gpu.add_rms_norm_backward(e, e, torch.ones(64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and dw.cpu().tolist() == [0.0] * 64
    n = gpu.add_rms_norm(e, torch.ones(64, dtype=torch.bfloat16, device="cuda"), residual=e, out_dtype=torch.int8)
    assert n.y.shape == (0, 64) and n.scale.shape == (0,) and n.h.shape == (0, 64)


# ------------------------------------------------------------------ the product with its epilogue

def act64(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def check_epilogue(gpu, M, N, K, ind, outd, act, bias=None, res=None, pre=False, scales=False, seed=0, offset=0, xw=None):
    """One call, every entry: the fp32 sums themselves are the plain product's (checked against the oracle elsewhere), from
    the same tiles (else sums of the same terms in another order); what follows them is computed here in 64 bits."""
    say("linear", M, N, K, ind, outd, act, "bias", bias, "res", res, "pre", pre, "scales", scales, "seed", seed)
    if ind == "i8":
        x, w = (torch.randint(-128, 128, s, generator=gen(seed + i), dtype=torch.int8) for i, s in enumerate(((M, K), (N, K))))
    else:
        t = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}.get(ind) or DT[ind]
        x, w = randn(seed, M, K).to(t), randn(seed + 1, N, K, std=K ** -0.5 if K else 1.0).to(t)
    g = lambda t: None if t is None else t.cuda()
    b = randn(seed + 2, N, dtype=DT[bias]) if bias else None
    r = randn(seed + 3, M, N, dtype=DT[res]) if res else None
    xs = torch.rand(M, generator=gen(seed + 4)) + 0.5 if scales else None
    ws = (torch.rand(N, generator=gen(seed + 5)) + 0.5) * (1 / (74 * 74 * max(K, 1) ** 0.5) if ind == "i8" else 1) if scales else None
    y, untouched = guarded((M, N), DT[outd], offset=offset)
    got = gpu.linear(x.cuda(), w.cuda(), bias=g(b), activation=act, residual=g(r), x_scale=g(xs), weight_scale=g(ws), out=y,
                     out_dtype=DT[outd], save_preact=pre)
    untouched()
    if K == 0:
        s = torch.zeros(M, N, dtype=torch.double)
    else:
        s = gpu.mm_bt(x.cuda(), w.cuda(), out_dtype=torch.int32 if ind == "i8" else torch.float32).cpu().double()
    z = s
    tol = u * s.abs() if ind == "i8" else torch.zeros_like(s)
    if ind in DT:
        c = {"bf16": gpu.BF16, "f16": gpu.F16}[ind]
        if gpu.gemm_bt_plan_epi(M, N, K, c, gpu.F32).as_dict() != gpu.gemm_bt_plan_ws(M, N, K, c, gpu.F32).as_dict():
            tol = 2 * K * u * (x.double().abs() @ w.double().abs().t())
    if scales:
        z = z * xs.double()[:, None] * ws.double()
        tol = tol * xs.double()[:, None] * ws.double() + 2 * u * z.abs()
    if b is not None:
        z = z + b.double()
        tol = tol + u * z.abs()
    if pre:
        close(got[1], z, tol, "preact")
    a = act64(z, act)
    tol = 1.13 * tol + (0 if act == "none" else 2.0 ** -20 * z.abs())
    if r is not None:
        a = a + r.double()
        tol = tol + u * a.abs()
    close(y, a, tol, "y")
    return y


# (M, N, K): every tile shape of the 16-bit kernels, ragged edges, K tails, odd rows of C
SHAPES16 = [(1, 1, 1), (1, 64, 64), (1, 4100, 2048), (16, 8192, 1000), (7, 5001, 333), (2, 1000, 8200), (16, 512, 8190), (3, 9, 17), (16, 200, 520), (16, 33, 4097), (17, 33, 65), (24, 4096, 8192), (31, 63, 127),
            (64, 64, 64), (64, 4100, 8192), (100, 2050, 134), (130, 264, 73), (257, 513, 129), (300, 700, 1000),
            (512, 512, 16384), (1024, 1024, 16384), (520, 1000, 16392), (700, 3200, 130), (1000, 1000, 136), (1000, 2999, 72), (1000, 3000, 136),
            (1000, 3000, 128), (1030, 1030, 202), (2000, 4000, 192), (2048, 1536, 72), (2048, 4004, 72), (3000, 1000, 72),
            (3000, 1000, 128), (4096, 4096, 130), (4100, 4100, 136), (4352, 4096, 64), (700, 2000, 1000), (1024, 4096, 128),
            (1213, 91, 4279), (100, 64, 4096), (300, 333, 8192), (65, 1000, 3000)]


def options(i):
    """A spread over what an epilogue may hold, for the i-th shape."""
    return dict(outd=("bf16", "f32", "f16")[i % 3], act=ACTS[(i // 2) % 5], bias=("own", None, "f32", "bf16", "f16")[i % 5],
                res=(None, "f32", "bf16", "f16")[(i // 3) % 4], pre=i % 2 == 0, scales=i % 4 == 3, offset=i % 2)


@pytest.mark.parametrize("n,shape", list(enumerate(SHAPES16)))
def test_linear_shapes(gpu, n, shape):
    for i in (n, n + 7, n + 31):
        ind = ("bf16", "f16")[(n + i) % 2]
        o = options(i)
        o["bias"] = ind if o["bias"] == "own" else o["bias"]
        check_epilogue(gpu, *shape, ind, seed=n, **o)


def test_linear_covers_every_kernel(gpu):
    """The shapes above plan each tile shape, and the forms split along K."""
    seen = set()
    for M, N, K in SHAPES16:
        p = gpu.gemm_bt_plan_epi(M, N, K, gpu.BF16, gpu.F32)
        parts = [p]
        if p.split_rows:
            parts.append(gpu.gemm_bt_plan_epi(M - p.split_rows, N, K, gpu.BF16, gpu.F32))
        seen |= {(q.kernel, q.variant, q.split_tiles > 0) for q in parts}
    assert {v for k, v, s in seen if k == 4 and not s} == {0, 1, 2, 6, 7, 8, 9, 12, 13, 14, 15}, seen
    assert {v for k, v, s in seen if k == 4 and s} == {1, 10, 11, 12}, seen
    assert any(k == 3 for k, _, _ in seen)


@pytest.mark.parametrize("ind", ["e4m3", "e5m2", "i8"])
@pytest.mark.parametrize("shape", [(1, 1, 16), (1, 72, 4096), (33, 65, 144), (130, 264, 208), (700, 1100, 128), (2050, 2050, 64),
                                   (2048, 4352, 80), (4100, 4096, 48), (4096, 4097, 32)])
def test_linear_eight_bits(gpu, ind, shape):
    n = sum(shape)
    for i in (n, n + 1, n + 5):
        o = options(i)
        o["bias"] = "bf16" if o["bias"] == "own" else o["bias"]
        o["scales"] = ind == "i8" or i % 2 == 0
        check_epilogue(gpu, *shape, ind, seed=n, **o)


@pytest.mark.parametrize("ind", ["e4m3", "e5m2", "i8"])
@pytest.mark.parametrize("shape", [(16, 8192, 512), (1, 4104, 4096), (5, 6001, 272), (64, 512, 8192), (33, 4096, 4096), (200, 300, 8208),
                                   (7, 70, 16384), (129, 1000, 4112)])
def test_linear_eight_bits_thin(gpu, ind, shape):
    """8-bit products of few rows: streaming, and cut along K (whose sums are those of other tiles, in another order)."""
    M, N, K = shape
    code = {"e4m3": gpu.FP8_E4M3, "e5m2": gpu.FP8_E5M2, "i8": gpu.INT8}[ind]
    p = gpu.gemm_bt_plan_epi(M, N, K, code, gpu.BF16)
    assert p.kernel == 3 if M <= 16 and N > 4096 else p.split_tiles > 0, p.as_dict()
    n = sum(shape)
    say("thin", ind, shape)
    t = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}.get(ind)
    if ind == "i8":
        x, w = (torch.randint(-128, 128, s, generator=gen(n + i), dtype=torch.int8) for i, s in enumerate(((M, K), (N, K))))
    else:
        x, w = randn(n, M, K).to(t), randn(n + 1, N, K).to(t)
    b, r = randn(n + 2, N, dtype=torch.bfloat16), randn(n + 3, M, N)
    xs, ws = torch.rand(M, generator=gen(n + 4)) + 0.5, (torch.rand(N, generator=gen(n + 5)) + 0.5) * K ** -0.5 * (2.0 ** -12 if ind == "i8" else 1)
    y, untouched = guarded((M, N), torch.float32)
    gpu.linear(x.cuda(), w.cuda(), bias=b.cuda(), activation="silu", residual=r.cuda(), x_scale=xs.cuda(), weight_scale=ws.cuda(),
               out=y, out_dtype=torch.float32)
    untouched()
    x64, w64 = x.float().double(), w.float().double()
    s, size = x64 @ w64.t(), x64.abs() @ w64.abs().t()
    scale = xs.double()[:, None] * ws.double()
    z = s * scale + b.double()
    tol = (u * s.abs() if ind == "i8" else K * u * size) * scale + 3 * u * (s * scale).abs() + u * z.abs()
    a = act64(z, "silu") + r.double()
    close(y, a, 1.13 * tol + 2.0 ** -20 * z.abs() + u * a.abs(), "y")
    if ind == "i8":  # whole numbers: every sum exact, in any order
        got = gpu.linear(x.cuda(), w.cuda(), out_dtype=torch.float32)
        assert torch.equal(got.cpu(), s.float())


def test_linear_every_term(gpu):
    """Each activation, output type, bias, residual and pre-activation at a ragged size."""
    for act, outd in itertools.product(ACTS, DT):
        check_epilogue(gpu, 77, 141, 96, "bf16", outd, act, bias="f16", res="bf16", pre=True, seed=1)
        check_epilogue(gpu, 9, 141, 96, "f16", outd, act, bias="bf16", res="f32", pre=True, scales=True, seed=2)
    for outd in DT:
        check_epilogue(gpu, 300, 260, 64, "bf16", outd, "none", seed=3)
    # no terms at all, where the plain product and the one with an epilogue are planned alike and where they are not
    for M, N, K in ((1, 64, 64), (16, 512, 8200), (64, 300, 8192), (512, 1024, 32768), (1024, 1024, 16384), (1213, 91, 4279),
                    (100, 64, 4096), (4352, 4096, 64)):
        check_epilogue(gpu, M, N, K, "bf16", "bf16", "none", seed=4)


def test_linear_empty_sums_and_no_rows(gpu):
    for M, N in ((5, 7), (300, 700), (1, 1)):
        for act in ACTS:
            check_epilogue(gpu, M, N, 0, "bf16", "f32", act, bias="bf16", res="f32", pre=True, scales=True, seed=4)
            check_epilogue(gpu, M, N, 0, "i8", "bf16", act, bias="bf16", seed=5)
    w = torch.ones(8, 16, dtype=torch.bfloat16, device="cuda")
    assert gpu.linear(w[:0], w).shape == (0, 8)
    assert gpu.linear(w, w[:0]).shape == (8, 0)
    assert gpu.linear(w.view(2, 4, 16), w, bias=w[0, :8].contiguous()).shape == (2, 4, 8)
    assert gpu.linear(w[0], w).shape == (8,)


def test_linear_in_place_residual(gpu):
    for M, N, K in ((16, 300, 64), (200, 333, 128), (4352, 4096, 64), (300, 64, 20000)):
        x, w, r = randn(1, M, K, dtype=torch.bfloat16).cuda(), randn(2, N, K, std=K ** -0.5, dtype=torch.bfloat16).cuda(), randn(3, M, N, dtype=torch.bfloat16).cuda()
        want = gpu.linear(x, w, activation="silu", residual=r)
        got = gpu.linear(x, w, activation="silu", residual=r, out=r)
        assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


def test_linear_large_offsets(gpu):
    """Results past 2^31 bytes from the start of C, of the residual and of the pre-activation: rows at both ends."""
    M, N, K = 270000, 4100, 32
    say("linear", M, N, K)
    x, w = randn(1, M, K, dtype=torch.bfloat16).cuda(), randn(2, N, K, dtype=torch.bfloat16).cuda()
    r = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    r[-300:] = 1.0
    y, z = gpu.linear(x, w, activation="relu", residual=r, save_preact=True)
    for rows in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        z64 = x[rows].double().cpu() @ w.double().cpu().t()
        tol = K * u * (x[rows].double().cpu().abs() @ w.double().cpu().abs().t())
        close(z[rows], z64, tol, "preact")
        y64 = z64.clamp_min(0) + r[rows].double().cpu()
        close(y[rows], y64, tol + u * y64.abs(), "y")


def test_linear_non_finite(gpu):
    """Infinities and NaN stay in their rows and columns, through each activation."""
    M, N, K = 40, 70, 64
    x, w, b, r = randn(1, M, K), randn(2, N, K, std=0.1), randn(3, N), randn(4, M, N)
    x[3, 5] = float("nan")
    b[7] = float("inf")
    b[8] = -3e38
    r[9, 9] = float("nan")
    x, w = x.bfloat16(), w.bfloat16()
    for act in ACTS:
        y = gpu.linear(x.cuda(), w.cuda(), bias=b.cuda(), activation=act, residual=r.cuda(), out_dtype=torch.float32).cpu()
        bad = torch.zeros(M, N, dtype=torch.bool)
        bad[3], bad[9, 9] = True, True
        assert torch.equal(torch.isnan(y), bad), act
        fine = ~bad[:, 7]
        assert bool((y[fine, 7] == float("inf")).all()), act
        if act != "none":
            assert bool((y[~bad[:, 8], 8].double() - r[~bad[:, 8], 8].double()).abs().max() <= 1e-6), act


# ------------------------------------------------------------------ the product, backward

def slope64(z, act):
    z = z.clone().requires_grad_(True)
    act64(z, act).sum().backward()
    return z.grad


@pytest.mark.parametrize("n", [1, 8, 9, 63, 64, 100, 200, 256, 300, 511, 520, 1000, 4096])
def test_act_backward(gpu, n):
    """dz and the bias gradient, through linear_backward without its products and through the C call for odd widths."""
    import ctypes

    lib = gpu.load()
    codes = {torch.float32: gpu.F32, torch.float16: gpu.F16, torch.bfloat16: gpu.BF16}
    for rows, dt, act in itertools.product((1, 6, 333), ("bf16", "f16", "f32"), ACTS):
        dy, z = randn(n + rows, rows, n, dtype=DT[dt]), randn(n + rows + 1, rows, n, std=2.5, dtype=DT[dt])
        zt = torch.float32 if (rows + n) % 2 else DT[dt]
        bt = DT[dt] if rows % 2 else torch.float32
        z = z.to(zt)
        say("act backward", rows, n, dt, act, zt, bt)
        need = ctypes.c_size_t()
        assert lib.gemm_bt_act_backward_workspace(rows, n, ctypes.byref(need)) == gpu.OK
        ws, ws_ok = guarded((need.value,), torch.uint8)
        dz, dz_ok = guarded((rows, n), DT[dt], offset=n % 2)
        db, db_ok = guarded((n,), bt)
        gdy, gz = dy.cuda(), z.cuda()
        st = lib.gemm_bt_act_backward(gdy.data_ptr(), gz.data_ptr(), dz.data_ptr(), db.data_ptr(), rows, n,
                                      ACTS.index(act), codes[DT[dt]], codes[zt], codes[bt], ws.data_ptr(), need.value,
                                      torch.cuda.current_stream().cuda_stream)
        assert st == gpu.OK
        for ok in (ws_ok, dz_ok, db_ok):
            ok()
        z64, dy64 = z.double(), dy.double()
        slope = slope64(z64, act)
        tol = dy64.abs() * (0 if act == "none" else 2.0 ** -20 * (1 + z64.abs() ** 3)) + u * (dy64 * slope).abs()
        close(dz, dy64 * slope, tol, ("dz", rows, n, dt, act))
        close(db, (dy64 * slope).sum(0), tol.sum(0) + (rows + 4) * u * (dy64 * slope).abs().sum(0), ("db", rows, n, dt, act))
        if rows == 6:  # too little workspace; in place of dy; no bias
            assert lib.gemm_bt_act_backward(gdy.data_ptr(), gz.data_ptr(), dz.data_ptr(), db.data_ptr(), rows, n, 1,
                                            codes[DT[dt]], codes[zt], codes[bt], ws.data_ptr(), need.value - 4,
                                            None) == gpu.ERR_INVALID_VALUE
            assert lib.gemm_bt_act_backward(gdy.data_ptr(), gz.data_ptr(), gdy.data_ptr(), None, rows, n, ACTS.index(act),
                                            codes[DT[dt]], codes[zt], codes[bt], None, 0,
                                            torch.cuda.current_stream().cuda_stream) == gpu.OK
            assert torch.equal(gdy, dz)


def check_backward(gpu, M, N, K, dt, act, bias=True, seed=0):
    say("linear backward", M, N, K, dt, act, "seed", seed)
    x, w = randn(seed, M, K, dtype=DT[dt]), randn(seed + 1, N, K, std=max(K, 1) ** -0.5, dtype=DT[dt])
    dy, z = randn(seed + 2, M, N, std=0.1, dtype=DT[dt]), randn(seed + 3, M, N, std=1.5, dtype=DT[dt])
    got = gpu.linear_backward(dy.cuda(), x.cuda(), w.cuda(), preact=z.cuda() if act != "none" else None, activation=act,
                              bias_grad=bias)
    x, w, dy, z = (t.double().cuda() for t in (x, w, dy, z))
    slope = slope64(z.cpu(), act).cuda()
    dz = dy * slope
    dz_tol = torch.zeros_like(dz)
    if act != "none":  # dz is rounded into the input's type before the products
        dz_tol = dy.abs() * 2.0 ** -20 * (1 + z.abs() ** 3) + u * dz.abs()
        dz_tol = dz_tol + UNIT[DT[dt]] * (dz.abs() + dz_tol) + TINY[DT[dt]]
    size = dz.abs() + dz_tol
    close(got.dx, (dz @ w).cpu(), (dz_tol @ w.abs() + N * u * (size @ w.abs())).cpu(), "dx")
    close(got.dweight, torch.mm(dz.t().contiguous(), x).cpu(),
          (torch.mm(dz_tol.t().contiguous(), x.abs()) + M * u * torch.mm(size.t().contiguous(), x.abs())).cpu(), "dw")
    if bias:
        tol = dy.abs() * 2.0 ** -20 * (1 + z.abs() ** 3) if act != "none" else torch.zeros_like(dz)
        close(got.dbias, dz.sum(0).cpu(), (tol.sum(0) + (M + 8) * u * dz.abs().sum(0)).cpu(), "db")
    else:
        assert got.dbias is None


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (5, 64, 72), (17, 8, 512), (100, 256, 264), (333, 1000, 520), (1000, 512, 2048),
                                   (2049, 1024, 72), (257, 4096, 1024),
                                   # rows that are not whole 16-byte chunks: N, K or both
                                   (1, 1, 1), (33, 9, 7), (64, 100, 130), (200, 1001, 64), (200, 64, 1001), (511, 2050, 333),
                                   # 256 x 256 tiles; sums cut into slices, of either product and of both
                                   (2048, 2048, 2050), (4096, 4096, 128), (5000, 64, 200), (70, 5000, 136), (9000, 513, 520),
                                   (100, 9000, 264), (6000, 6000, 128), (40000, 520, 512)])
def test_linear_backward(gpu, M, N, K):
    for i, (dt, act) in enumerate(itertools.product(("bf16", "f16"), ACTS)):
        if (M + i) % 2 == 0 and (M * N * K < 1e8 or i in (1, 2, 8)) or M < 100:
            check_backward(gpu, M, N, K, dt, act, bias=i % 3 != 0, seed=M + i)


def test_linear_backward_slices_are_planned(gpu):
    """The sizes above include products cut along their sums: the workspace holds their fp32 slices."""
    import ctypes

    n = ctypes.c_size_t()
    size = lambda M, N, K: (gpu.load().gemm_bt_linear_backward_workspace(M, N, K, 0, ctypes.byref(n)), n.value)[1]
    # besides the slices: partial sums of the bias, at most one row per row of dy
    for M, N, K, result in ((5000, 64, 200, 64 * 200), (40000, 520, 512, 520 * 512)):   # dw = a sum over M
        assert size(M, N, K) >= 2 * result * 4 + 4 * N
    for M, N, K, result in ((70, 5000, 136, 70 * 136), (100, 9000, 264, 100 * 264)):     # dx = a sum over N
        assert size(M, N, K) >= 2 * result * 4 + 4 * N
    assert size(4096, 4096, 4096) <= 4096 * 4 * 4096  # not cut


def test_linear_backward_parts_and_places(gpu):
    """Each gradient alone, inputs that start off a 16-byte boundary, leading dimensions; the same bits on every run."""
    for M, N, K in ((70, 96, 130), (300, 512, 256), (5000, 64, 200)):
        dy, x, w, z = (randn(i, *s, std=0.3, dtype=torch.bfloat16).cuda() for i, s in enumerate(((M, N), (M, K), (N, K), (M, N))))
        for act in ("none", "silu"):
            p = z if act != "none" else None
            whole = gpu.linear_backward(dy, x, w, preact=p, activation=act)
            again = gpu.linear_backward(dy, x, w, preact=p, activation=act)
            assert all(torch.equal(a, b) for a, b in zip(whole, again))
            for i, kw in enumerate((dict(bias_grad=False, need_dweight=False), dict(bias_grad=False, need_dx=False),
                                    dict(need_dx=False, need_dweight=False))):
                part = gpu.linear_backward(dy, x, w, preact=p, activation=act, **kw)
                assert torch.equal(part[i], whole[i]) and [g is None for g in part] == [j != i for j in range(3)]
            off = []
            for t in (dy, x, w, z):
                buf = torch.zeros(t.numel() + 3, dtype=t.dtype, device="cuda")
                buf[3:] = t.flatten()
                off.append(buf[3:].view(t.shape))
            moved = gpu.linear_backward(off[0], off[1], off[2], preact=off[3] if p is not None else None, activation=act)
            assert all(torch.equal(a, b) for a, b in zip(whole, moved))
            cube = gpu.linear_backward(dy.view(2, M // 2, N), x.view(2, M // 2, K), w, preact=None if p is None else p.view(2, M // 2, N),
                                       activation=act)
            assert cube.dx.shape == (2, M // 2, K) and torch.equal(cube.dx.view(M, K), whole.dx) and torch.equal(cube.dweight, whole.dweight)


def test_linear_gradient_against_differences(gpu):
    """dx, dw, db of L = sum(y * dy) against central differences of the 64-bit forward pass, for inputs that 16 bits hold
    exactly; what the kernels round is dz and the results, 2^-8 relative each, and the kept pre-activation."""
    M, N, K = 6, 16, 24
    x, w, dy = (randn(50 + i, *s, dtype=torch.bfloat16) for i, s in enumerate(((M, K), (N, K), (M, N))))
    w = (w * 0.25).bfloat16()
    b = randn(60, N, dtype=torch.bfloat16)
    for act in ACTS[2:]:
        y, z = gpu.linear(x.cuda(), w.cuda(), bias=b.cuda(), activation=act, save_preact=True)
        got = gpu.linear_backward(dy.cuda(), x.cuda(), w.cuda(), preact=z, activation=act)

        def loss(x, w, b):
            return (act64(x @ w.t() + b, act) * dy.double()).sum()

        args = [x.double(), w.double(), b.double()]
        step = 1e-5
        for t, grad in ((0, got.dx), (1, got.dweight), (2, got.dbias)):
            for at in ((0, 0), (3, 11), (5, 15)):
                at = at if t != 2 else at[1:]
                e = torch.zeros_like(args[t])
                e[at] = step
                up, down = [a + e if i == t else a for i, a in enumerate(args)], [a - e if i == t else a for i, a in enumerate(args)]
                want = float((loss(*up) - loss(*down)) / (2 * step))
                # 24 terms of size up to |dy| |w|: three roundings of 2^-8 on sums of magnitudes
                size = float((dy.double().abs().amax() * args[1 - t].abs().amax() if t < 2 else dy.double().abs().amax()) * 6)
                assert abs(float(grad[at]) - want) <= 3 * 2.0 ** -8 * size, (act, t, at, float(grad[at]), want)


def test_linear_backward_refusals(gpu):
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        gpu.linear_backward(dy, x, w, activation="gelu")               # no pre-activation
    with pytest.raises(ValueError):
        gpu.linear_backward(dy, x, w, activation="swish")
    with pytest.raises(TypeError):
        gpu.linear_backward(dy.float(), x, w)
    with pytest.raises(ValueError):
        gpu.linear_backward(dy[:, :7], x, w)
    with pytest.raises(ValueError):
        gpu.linear(x, w, bias=torch.zeros(9, device="cuda"))
    with pytest.raises(ValueError):
        gpu.linear(x, w, residual=x)
    with pytest.raises(ValueError):
        gpu.linear(x, w, x_scale=torch.ones(5, device="cuda"))
    with pytest.raises(TypeError):
        gpu.linear(x.float(), w.float())
    with pytest.raises(TypeError):
        gpu.linear(x, w, out_dtype=torch.int32)
    with pytest.raises(ValueError):
        gpu.add_rms_norm(x, torch.ones(15, device="cuda"))
    with pytest.raises(TypeError):
        gpu.add_rms_norm(x, torch.ones(16, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        gpu.add_rms_norm(x, torch.ones(16, device="cuda"), residual=x[:3])
    with pytest.raises(TypeError):
        gpu.quantize_rows(x, torch.float8_e5m2)
    with pytest.raises(gpu.GemmBtError):
        gpu.add_rms_norm(x, torch.ones(16, device="cuda"), eps=-1.0)
    empty = gpu.linear_backward(dy[:0], x[:0], w)
    assert empty.dx.shape == (0, 16) and not bool(empty.dweight.any()) and not bool(empty.dbias.any())
    part = gpu.linear_backward(dy, x, w, bias_grad=False, need_dx=False)
    assert part.dx is None and part.dbias is None and part.dweight.shape == (8, 16)


# ------------------------------------------------------------------ streams, graphs, repetition

def block(gpu, t):
    """The operators as they are used together: a pre-norm feed-forward block, forward and backward, and its 8-bit form."""
    n = gpu.add_rms_norm(t["x"], t["g"], residual=t["r"], save_rstd=True)
    a, z = gpu.linear(n.y, t["w1"], bias=t["b1"], activation="gelu_tanh", save_preact=True)
    y = gpu.linear(a, t["w2"], residual=n.h)
    g2 = gpu.linear_backward(t["dy"], a, t["w2"], bias_grad=False)
    g1 = gpu.linear_backward(g2.dx, n.y, t["w1"], preact=z, activation="gelu_tanh")
    dx, dg = gpu.add_rms_norm_backward(g1.dx, n.h, t["g"], n.rstd, dh=t["dy"])
    q = gpu.add_rms_norm(t["x"], t["g"], residual=t["r"], out_dtype=torch.float8_e4m3fn)
    y8 = gpu.linear(q.y, t["q1"], x_scale=q.scale, weight_scale=t["s1"], activation="silu")
    qa = gpu.quantize_rows(y8, torch.int8)
    return [y, dx, dg, g1.dweight, g1.dbias, g2.dweight, q.y.view(torch.uint8), q.scale, y8, qa.q, qa.scale]


def block_inputs(gpu, rows=200, d=512, f=1024):
    t = {"x": randn(1, rows, d), "r": randn(2, rows, d), "g": 1 + randn(3, d, std=0.1), "w1": randn(4, f, d, std=d ** -0.5),
         "b1": randn(5, f, std=0.1), "w2": randn(6, d, f, std=f ** -0.5), "dy": randn(7, rows, d, std=0.1)}
    t = {k: v.bfloat16().cuda() for k, v in t.items()}
    t["q1"], t["s1"] = gpu.quantize_rows(t["w1"])
    return t


def test_streams(gpu):
    """On a stream that is not torch's current one, behind work that is still filling the inputs."""
    t = block_inputs(gpu)
    want = [o.clone() for o in block(gpu, t)]
    side = torch.cuda.Stream()
    for _ in range(3):
        late = {k: torch.empty_like(v) for k, v in t.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            busy = torch.randn(2048, 2048, device="cuda")
            for _ in range(10):
                busy = busy @ busy * 0.01
            for k, v in t.items():
                late[k].copy_(v)
            got = block(gpu, late)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_stream_argument(gpu):
    """``stream``: the copies that a call makes of strided inputs are in that stream's order too."""
    x0, w = randn(1, 64, 512, dtype=torch.bfloat16), randn(2, 256, 512, std=0.05, dtype=torch.bfloat16).cuda()
    r0, g = randn(3, 64, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    want = gpu.linear(x0.cuda(), w, activation="silu", residual=r0.cuda())
    wantn = gpu.add_rms_norm(want, g, residual=r0.cuda(), save_rstd=True)
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        xt = torch.empty(512, 64, dtype=torch.bfloat16, device="cuda")
        rt = torch.empty(256, 64, dtype=torch.bfloat16, device="cuda")
        xs, rs = x0.t().contiguous().cuda(), r0.t().contiguous().cuda()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            busy = torch.randn(2048, 2048, device="cuda")
            for _ in range(20):
                busy = busy @ busy * 0.01
            xt.copy_(xs)
            rt.copy_(rs)
        got = gpu.linear(xt.t(), w, activation="silu", residual=rt.t(), stream=handle)
        n = gpu.add_rms_norm(got, g, residual=rt.t(), save_rstd=True, stream=handle)
        q = gpu.quantize_rows(got, torch.int8, stream=handle)
        dx, dw = gpu.add_rms_norm_backward(got, n.h, g, n.rstd, dh=rt.t(), stream=handle)
        b = gpu.linear_backward(got, xt.t(), w, preact=got, activation="silu", stream=handle)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(n.y, wantn.y) and torch.equal(n.h, wantn.h)
        assert torch.equal(q.q, gpu.quantize_rows(want, torch.int8).q)
        wdx, wdw = gpu.add_rms_norm_backward(want, wantn.h, g, wantn.rstd, dh=r0.cuda())
        wb = gpu.linear_backward(want, x0.cuda(), w, preact=want, activation="silu")
        assert torch.equal(dx, wdx) and torch.equal(dw, wdw) and all(torch.equal(a, c) for a, c in zip(b, wb))


def test_graph_without_a_warm_up(gpu):
    """A product that is cut along K, captured before any call on that stream: its counters are the graph's own, whatever
    runs on the stream in between and in whichever order two graphs are replayed."""
    for dt in (torch.bfloat16, torch.int8):
        x, w = randn(1, 8, 8192, std=3.0).to(dt).cuda(), randn(2, 512, 8192, std=3.0).to(dt).cuda()
        code = {torch.bfloat16: gpu.BF16, torch.int8: gpu.INT8}[dt]
        assert gpu.gemm_bt_plan_epi(8, 512, 8192, code, gpu.BF16).split_tiles > 0
        want = gpu.linear(x, w)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graphs, outs = [], []
        for _ in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                outs.append(gpu.linear(x, w))
        with torch.cuda.stream(side):
            eager = gpu.linear(x, w)
        side.synchronize()
        assert torch.equal(eager, want)
        for i in (1, 0, 1, 1, 0):
            outs[i].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want), i
            with torch.cuda.stream(side):
                assert torch.equal(gpu.linear(x, w), want)


def test_graph_replays(gpu):
    t = block_inputs(gpu)
    want = [o.clone() for o in block(gpu, t)]
    other = {k: (v.float() * 0.5).to(v.dtype) if v.dtype == torch.bfloat16 else v.clone() for k, v in t.items()}
    fed = {k: v.clone() for k, v in t.items()}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block(gpu, fed)  # workspaces exist before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = block(gpu, fed)
    want2 = [o.clone() for o in block(gpu, other)]
    for inputs, expected in ((t, want), (other, want2), (t, want)):
        for k in fed:
            fed[k].copy_(inputs[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, expected))
        assert all(torch.equal(a, b) for a, b in zip(block(gpu, inputs), expected))  # eager work in between
