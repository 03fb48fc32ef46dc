"""The layer norm and its backward pass against plain implementations in 64 bits.

Where the tolerances come from (u = 2^-24, the unit roundoff of fp32).  A sum over a row of d entries passes at most 16 + 6 +
16 additions in a register, over a wave and over a workgroup, 8 more per 8192 entries past 16384: S = (60 + d/2048) u
relative to the sum of magnitudes, some roundings of its terms included.
  * centred values: c = (h - m0) - off, off the mean of h - m0.  h is one rounding of x + residual where there is one; m0
    is within S mean|h|, so the centred values are within 2 u (|h| + mean|h|) for that rounding (nothing without a
    residual) and S (|c| + mean|c|) for the rest, but for a term of second order, 2 S^2 mean|h|: EC;
  * mean: EC's average, and its own rounding;
  * rstd: half of the relative error of the variance: S, and rms(EC) / sqrt(var + eps);
  * y: rstd |w| EC, |c rstd w| (rstd's error + 4 u), and 2 u (|c rstd w| + |b|) for the sum; then one rounding into the
    stored type;
  * the backward pass: xhat is three roundings of (h - mean) rstd, the means S relative to the mean magnitudes of what
    they are taken of; sums over M rows are within (M + 8) u of the sum of magnitudes.
"""
import ctypes
import itertools
import math

import pytest
import torch

import dense_tiled_gemm_amd as gb
from test_layers_gpu import DT, EIGHT, QMAX, close, guarded, randn, say, u

BAD, UNSUP = gb.ERR_INVALID_VALUE, gb.ERR_UNSUPPORTED
EPS = 1e-5


def s_rel(d):
    return (60 + d / 2048) * u


def norm64(x, r, w, b, eps=EPS):
    """(h, mean, rstd, y) in 64 bits and the tolerances of each but h."""
    d = x.shape[-1]
    h = x.double() + (0 if r is None else r.double())
    mean = h.mean(-1, keepdim=True)
    c = h - mean
    var = (c * c).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    plain = c * rstd * w.double()
    y = plain + (0 if b is None else b.double())
    S, size = s_rel(d), h.abs().mean(-1, keepdim=True)
    ec = (0 if r is None else 2 * u * (h.abs() + size)) + S * (c.abs() + c.abs().mean(-1, keepdim=True)) + 2 * S * S * size
    t_mean = ec.mean(-1, keepdim=True) + u * mean.abs()
    t_rstd = S + (ec * ec).mean(-1, keepdim=True).sqrt() * rstd
    t_y = rstd * w.double().abs() * ec + plain.abs() * (t_rstd + 6 * u) + (0 if b is None else 2 * u * b.double().abs())
    return (h, mean[..., 0], rstd[..., 0], y), (t_mean[..., 0], (t_rstd * rstd)[..., 0], t_y)


def check_codes(q, scale, y64, tol, qt, what):
    """q and its scales against the exact rows y64, each known to within tol."""
    amax = y64.abs().amax(-1)
    s = scale.cpu().double()
    assert bool(((s * QMAX[qt] - torch.clamp(amax, min=2.0 ** -100 * QMAX[qt])).abs() <= tol.amax(-1) + 4 * u * amax).all()), what
    v, t = y64 / s[..., None], tol / s[..., None]
    top = (v.abs() + t) * (1 + 1e-6)  # a value that may lie past a power of two is rounded as there
    half = torch.full_like(v, 0.5) if qt == "i8" else torch.exp2(torch.floor(torch.log2(top.clamp_min(2.0 ** -6))) - 4)
    got = q.float().double().cpu()
    assert bool(((got - v).abs() <= half + t + 16 * u * v.abs()).all()), what
    assert bool((got.abs() <= QMAX[qt]).all()), what


def check(gpu, rows, d, dt, out, wt, res, bias, seed, mean=0.0, std=2.0):
    say("layer norm", rows, d, dt, out, wt, res, bias, "seed", seed)
    x = (randn(seed, rows, d, std=std) + mean).to(DT[dt])
    r = randn(seed + 1, rows, d, std=3.0, dtype=DT[dt]) if res else None
    w_dt = DT[dt] if wt == "own" else torch.float32
    w = (1 + randn(seed + 2, d, std=0.3)).to(w_dt)
    b = randn(seed + 3, d, std=0.5).to(w_dt) if bias else None
    y, untouched = guarded((rows, d), EIGHT.get(out, DT[dt]), offset=seed % 3)
    got = gpu.add_layer_norm(x.cuda(), w.cuda(), None if b is None else b.cuda(), residual=None if r is None else r.cuda(), eps=EPS,
                             out_dtype=y.dtype, save_stats=True, out=y)
    untouched()
    (h, m, rstd, y64), (t_mean, t_rstd, t_y) = norm64(x, r, w, b)
    close(got.mean, m, t_mean, "mean")
    close(got.rstd, rstd, t_rstd, "rstd")
    if res:
        close(got.h, h, 2 * u * h.abs(), "h")
    else:
        assert got.h is None
    if out == "own":
        assert got.scale is None
        close(got.y, y64, t_y, "y")
    else:
        check_codes(got.y, got.scale, y64, t_y, out, (rows, d, dt, out))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [1, 2, 7, 8, 9, 63, 64, 130, 512, 513, 1000, 1024, 1031, 2048, 2049, 2056, 4096, 4097, 8192, 8200, 16384])
def test_layer_norm(gpu, d):
    for i, (rows, dt, out, res) in enumerate(itertools.product((1, 3, 5) if d > 600 else (1, 7, 1200), DT, ("own", "e4m3", "i8"), (0, 1))):
        if (i + d) % 2 and d > 9:  # half of the combinations at each width
            continue
        check(gpu, rows, d, dt, out, ("own", "f32")[i // 2 % 2], res, i // 3 % 2, 1000 * d + rows)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(515, 4096), (513, 8192), (600, 3000), (700, 1500), (520, 12000), (2100, 700), (1300, 257), (2, 16392),
                                    (3, 33001), (1, 100003)])
def test_many_and_long_rows(gpu, rows, d):
    for dt, out, res in (("bf16", "own", 1), ("f32", "e4m3", 1), ("f16", "i8", 0), ("f32", "own", 0)):
        check(gpu, rows, d, dt, out, "own", res, 1, rows + d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [5, 64, 1000, 4097, 20000])
def test_rows_far_from_zero(gpu, d):
    """Rows whose mean is far above their spread: the mean's rounding must not show in what is left."""
    for dt, mean, std in (("f32", 1000.0, 1.0), ("f32", -3e5, 2.0), ("f32", 1e6, 0.5), ("f16", 500.0, 1.0), ("bf16", 64.0, 1.0)):
        check(gpu, 6, d, dt, "own", "own", 0, 1, d, mean, std)
    # rows of one value: their mean is that value, and next to nothing is left
    x = torch.tensor([0.0, 1.0, 1 / 3, -1e5, 123456.789, -2.0 ** -100])[:, None].expand(6, d).contiguous()
    w, b = torch.ones(d), randn(1, d)
    got = gpu.add_layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS, save_stats=True)
    (_, _, rstd, y64), (_, t_rstd, t_y) = norm64(x, None, w, b)
    assert torch.equal(got.mean.cpu(), x[:, 0])
    close(got.rstd, rstd, t_rstd, "rstd")
    close(got.y, y64, t_y, "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("d", [3, 40, 2048, 20000])
def test_extremes(gpu, d, dt):
    """Rows of the type's largest values and rows with an infinity or a NaN: each row by itself."""
    big = torch.finfo(DT[dt]).max
    x = randn(3, 8, d)
    x[0] = big / 4 if dt != "f32" else 2.0 ** 100
    x[1] = big / 4
    x[1, ::2] = -big / 4
    x[2] = big
    x[3, d // 2] = float("inf")
    x[4, d - 1] = float("nan")
    x[5, 0] = -float("inf")
    x[6] *= 2.0 ** -20
    x = x.to(DT[dt])
    w, b = torch.ones(d), torch.zeros(d)
    say("layer norm extremes", d, dt)
    got = gpu.add_layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS, save_stats=True, out_dtype=torch.float32)
    (_, mean, rstd, y64), (t_mean, t_rstd, t_y) = norm64(x, None, w, b)
    assert bool(torch.isnan(got.y[[3, 4, 5]]).all())
    for row in (0, 1, 2, 6, 7):
        close(got.mean[row], mean[row], t_mean[row] + 2.0 ** -100, ("mean", row))
        close(got.rstd[row], rstd[row], t_rstd[row], ("rstd", row))
        close(got.y[row], y64[row], t_y[row], ("y", row))
    for qt in EIGHT:
        n = gpu.add_layer_norm(x.cuda(), w.cuda(), out_dtype=EIGHT[qt])
        assert bool(torch.isnan(n.scale[[3, 4, 5]]).all()) and bool(torch.isfinite(n.scale[[0, 1, 2, 6, 7]]).all())


@pytest.mark.gpu
def test_layouts_and_places(gpu):
    wide = randn(5, 40, 700, dtype=torch.bfloat16).cuda()
    w, b = (1 + randn(6, 333, std=0.2)).cuda(), randn(7, 333).cuda()
    for x in (wide[:, 3:336], wide[::2, 64:397], wide[1:, :333], wide.t()[:333].t()[:, :333]):
        r = wide[:x.shape[0], 350:683]
        (_, _, _, y64), (_, _, t_y) = norm64(x.cpu(), r.cpu(), w.cpu(), b.cpu())
        close(gpu.add_layer_norm(x, w, b, residual=r).y, y64, t_y, "strided")
    cube = randn(7, 4, 5, 96, dtype=torch.float16).cuda()
    w96 = torch.ones(96, dtype=torch.float16, device="cuda")
    for x in (cube, cube.transpose(0, 1)):
        got = gpu.add_layer_norm(x, w96, residual=x, out_dtype=torch.float32, save_stats=True)
        (h, mean, _, y64), (t_mean, _, t_y) = norm64(x.cpu(), x.cpu(), w96.cpu(), None)
        assert got.y.shape == x.shape and got.rstd.shape == got.mean.shape == x.shape[:-1]
        close(got.y, y64, t_y, "cube")
        close(got.mean, mean, t_mean, "cube mean")
        close(got.h, h, 2 * u * h.abs(), "cube h")
    for d, out in itertools.product((64, 4096, 20000), (None, torch.float8_e4m3fn)):
        x, r, w = randn(8, 6, d, dtype=torch.bfloat16), randn(9, 6, d, dtype=torch.bfloat16), torch.ones(d, dtype=torch.bfloat16)
        (h, _, _, y64), (_, _, t_y) = norm64(x, r, w, None)
        for into in (0, 1):
            pair = [x.cuda(), r.cuda()]
            got = gpu.add_layer_norm(pair[0], w.cuda(), residual=pair[1], out_dtype=out, h_out=pair[into])
            assert got.h.data_ptr() == pair[into].data_ptr()
            close(pair[into], h, 2 * u * h.abs(), ("in place", d))
            assert torch.equal(pair[1 - into].cpu(), (x, r)[1 - into])
            if out is None:
                close(got.y, y64, t_y, ("in place y", d))
            else:
                check_codes(got.y, got.scale, y64, t_y, "e4m3", ("in place", d))


@pytest.mark.gpu
def test_no_rows_and_no_elements(gpu):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    got = gpu.add_layer_norm(z(0, 8), z(8), z(8), residual=z(0, 8), save_stats=True)
    assert got.y.shape == (0, 8) and got.mean.shape == (0,)
    got = gpu.add_layer_norm(z(3, 0), z(0), z(0), eps=0.25, out_dtype=torch.int8, save_stats=True)
    assert got.mean.tolist() == [0.0] * 3 and got.rstd.tolist() == [2.0] * 3 and got.scale.tolist() == [2.0 ** -100] * 3
    f = lambda *s: torch.zeros(*s, device="cuda")
    back = gpu.add_layer_norm_backward(z(0, 8), z(0, 8), z(8) + 1, f(0), f(0))
    assert back.dx.shape == (0, 8) and not bool(back.dweight.any()) and not bool(back.dbias.any())
    back = gpu.add_layer_norm_backward(z(3, 0), z(3, 0), z(0), f(3), f(3))
    assert back.dx.shape == (3, 0) and back.dweight.shape == back.dbias.shape == (0,)


# ------------------------------------------------------------------ backward

def back64(dy, h, w, mean, rstd, dh):
    dy, h, w, mean, rstd = dy.double(), h.double(), w.double(), mean.double()[..., None], rstd.double()[..., None]
    S = s_rel(dy.shape[-1])
    xhat, g = (h - mean) * rstd, dy * w
    avg = lambda t: t.mean(-1, keepdim=True)
    dx = rstd * (g - avg(g) - xhat * avg(g * xhat)) + (0 if dh is None else dh.double())
    t_dx = rstd * (8 * u * g.abs() + S * avg(g.abs()) + (S + 10 * u) * xhat.abs() * avg((g * xhat).abs())) + 2 * u * dx.abs()
    if dh is not None:
        t_dx = t_dx + 2 * u * dh.double().abs()
    flat = lambda t: t.flatten(0, -2)
    n = flat(dy).shape[0]
    return (dx, flat(dy * xhat).sum(0), flat(dy).sum(0)), \
        (t_dx, (n + 8) * u * flat(dy * xhat).abs().sum(0), (n + 8) * u * flat(dy).abs().sum(0))


def stats(h, eps=EPS):
    f = h.float()
    mean = f.mean(-1)
    return mean, torch.rsqrt((f - mean[..., None]).square().mean(-1) + eps)


def check_backward(gpu, rows, d, dt, wt, res, bias, seed):
    say("layer norm backward", rows, d, dt, wt, res, bias, "seed", seed)
    h, dy = (randn(seed, rows, d, std=2.0) + 0.5).to(DT[dt]), randn(seed + 1, rows, d, std=0.1, dtype=DT[dt])
    dh = randn(seed + 2, rows, d, std=0.1, dtype=DT[dt]) if res else None
    w = (1 + randn(seed + 3, d, std=0.3)).to(DT[dt] if wt == "own" else torch.float32)
    mean, rstd = stats(h)
    args = [t.cuda() for t in (dy, h, w, mean, rstd)]
    got = gpu.add_layer_norm_backward(*args, dh=None if dh is None else dh.cuda(), bias_grad=bool(bias))
    again = gpu.add_layer_norm_backward(*args, dh=None if dh is None else dh.cuda())
    want, tol = back64(dy, h, w, mean, rstd, dh)
    for g, a, want_g, t, what in zip(got, again, want, tol, ("dx", "dw", "db")):
        if g is None:
            assert what == "db" and not bias
            g = a
        assert torch.equal(g, a), what  # the same bits on every run, with and without dbias
        close(g, want_g, t, (what, rows, d, dt))
    assert got.dx.dtype == DT[dt] and got.dweight.dtype == w.dtype


@pytest.mark.gpu
@pytest.mark.parametrize("d", [1, 7, 8, 64, 100, 512, 520, 1000, 1031, 2048, 2050, 4096, 4099, 8192, 8200, 16384, 17001])
def test_backward(gpu, d):
    for i, (rows, dt, wt, res) in enumerate(itertools.product((1, 5, 300) if d <= 4096 else (1, 5), DT, ("own", "f32"), (0, 1))):
        if (i + i // 2 + d) % 2 and d > 8:
            continue
        check_backward(gpu, rows, d, dt, wt, res, i % 3, d + rows)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(3000, 200), (2500, 768), (1500, 2000), (1200, 4000), (700, 8000), (530, 10000), (1300, 505), (1100, 1021),
                                    (600, 2042), (530, 4099), (513, 9999), (2000, 2049)])
def test_backward_many_rows(gpu, rows, d):
    for dt, wt, res, bias in (("bf16", "own", 1, 1), ("f32", "own", 0, 0), ("f16", "f32", 1, 1)):
        check_backward(gpu, rows, d, dt, wt, res, bias, rows)


@pytest.mark.gpu
def test_backward_layouts_and_dx_in_dh(gpu):
    for rows, d in ((5, 96), (700, 333)):
        wide = [randn(i, rows, d + 5 + i, dtype=torch.bfloat16).cuda() for i in range(3)]
        dy, h, dh = (t[:, 2 + i:2 + i + d] for i, t in enumerate(wide))
        w = (1 + randn(9, d, std=0.3)).bfloat16().cuda()
        mean, rstd = stats(h)
        got = gpu.add_layer_norm_backward(dy, h, w, mean, rstd, dh=dh)
        want, tol = back64(dy.cpu(), h.cpu(), w.cpu(), mean.cpu(), rstd.cpu(), dh.cpu())
        for g, want_g, t in zip(got, want, tol):
            close(g, want_g, t, (rows, d))
        lib, need = gpu.load(), ctypes.c_size_t()
        assert lib.gemm_bt_layer_norm_backward_workspace(rows, d, ctypes.byref(need)) == gpu.OK
        ws = torch.empty(max(1, need.value), dtype=torch.uint8, device="cuda")
        there, dw, db = dh.contiguous(), torch.empty_like(w), torch.empty_like(w)
        call = lambda dx, n: lib.gemm_bt_layer_norm_backward(
            dy.data_ptr(), dy.stride(0), h.data_ptr(), h.stride(0), w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), there.data_ptr(), d,
            dx, dw.data_ptr(), db.data_ptr(), rows, d, gpu.BF16, gpu.BF16, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        if need.value:
            assert call(there.data_ptr(), need.value - 1) == BAD
        assert call(dy.data_ptr(), need.value) == BAD and call(h.data_ptr(), need.value) == BAD
        assert call(there.data_ptr(), need.value) == gpu.OK
        assert torch.equal(there, got.dx) and torch.equal(dw, got.dweight) and torch.equal(db, got.dbias)


@pytest.mark.gpu
def test_gradient_against_differences(gpu):
    """sum(y * dy + h * dh) moved along a random direction, against the gradients along it."""
    rows, d, step = 6, 50, 1e-4
    x, r, dy, dh, vx = (randn(i, rows, d).double() for i in range(5))
    w, b, vw, vb = (1 + randn(7, d).double() * 0.3), randn(8, d).double(), randn(9, d).double(), randn(10, d).double()

    def loss(t):
        h, _, _, y = norm64(x + t * vx, r, w + t * vw, b + t * vb)[0]
        return float((y * dy + h * dh).sum())
    f = lambda t: t.float().cuda()
    n = gpu.add_layer_norm(f(x), f(w), f(b), residual=f(r), eps=EPS, save_stats=True)
    g = gpu.add_layer_norm_backward(f(dy), n.h, f(w), n.mean, n.rstd, dh=f(dh))
    along = sum(float((a.double().cpu() * v).sum()) for a, v in zip(g, (vx, vw, vb)))
    want = (loss(step) - loss(-step)) / (2 * step)
    # the gradients' own errors, below 2^-16 of each term, and the differences' third order
    size = sum(float((a.double().cpu() * v).abs().sum()) for a, v in zip(g, (vx, vw, vb)))
    assert abs(along - want) <= 2.0 ** -16 * size + 1e-4 * abs(want), (along, want)


@pytest.mark.gpu
def test_streams_and_graphs(gpu):
    """A captured forward and backward pass replayed with other inputs and eager work in between, on a side stream."""
    rows, d = 700, 1000
    make = lambda seed: [randn(seed, rows, d, dtype=torch.bfloat16).cuda(), randn(seed + 1, rows, d, dtype=torch.bfloat16).cuda(),
                         (1 + randn(seed + 2, d, std=0.2)).bfloat16().cuda(), randn(seed + 3, d).bfloat16().cuda(),
                         randn(seed + 4, rows, d, std=0.1, dtype=torch.bfloat16).cuda()]

    def both(x, r, w, b, dy, stream=None):
        n = gpu.add_layer_norm(x, w, b, residual=r, save_stats=True, stream=stream)
        return [n.y, n.h, n.mean, n.rstd, *gpu.add_layer_norm_backward(dy, n.h, w, n.mean, n.rstd, dh=dy, stream=stream)]
    one, two = make(1), make(11)
    want = [both(*one), both(*two)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        got = both(*one, stream=handle)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    fed = [t.clone() for t in one]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = both(*fed)
    for i in (0, 1, 0, 1):
        for t, v in zip(fed, (one, two)[i]):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
        assert all(torch.equal(a, b) for a, b in zip(both(*(one, two)[1 - i]), want[1 - i]))


# ------------------------------------------------------------------ refusals

def norm(x=16, ldx=8, res=None, ldr=0, w=16, b=16, y=16, h=None, scale=None, mean=None, rstd=None, rows=2, d=8, eps=1e-6, xt=gb.BF16,
         wt=gb.BF16, yt=gb.BF16):
    return int(gb.load().gemm_bt_layer_norm(x, ldx, res, ldr, w, b, y, h, scale, mean, rstd, rows, d, eps, xt, wt, yt, None))


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), BAD), (dict(d=-1), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(xt=gb.INT8), UNSUP), (dict(wt=gb.F16), UNSUP), (dict(xt=gb.F32, wt=gb.BF16), UNSUP), (dict(yt=gb.FP8_E5M2), UNSUP),
    (dict(d=2 ** 31 - 1, ldx=2 ** 31), UNSUP), (dict(rows=2 ** 31 + 1), UNSUP),
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(x=17), BAD), (dict(y=17), BAD), (dict(b=17), BAD),
    (dict(yt=gb.FP8_E4M3), BAD), (dict(yt=gb.INT8, scale=18), BAD), (dict(rstd=18), BAD), (dict(mean=18), BAD), (dict(h=17), BAD),
    (dict(wt=gb.F32, b=18), BAD), (dict(ldx=7), BAD), (dict(res=16, ldr=7), BAD), (dict(res=17, ldr=8), BAD),
    (dict(rows=0, x=None, w=None, y=None), gb.OK), (dict(d=0, x=None, w=None, y=None), gb.OK), (dict(d=0, mean=18), BAD),
])
def test_refusals(kw, want):
    assert norm(**kw) == want


def back(dy=16, h=16, w=16, mean=16, rstd=16, dh=None, dx=32, dw=16, db=16, rows=2, d=8, xt=gb.BF16, wt=gb.BF16, ws=16, n=1 << 20,
         ld=(8, 8, 8)):
    return int(gb.load().gemm_bt_layer_norm_backward(dy, ld[0], h, ld[1], w, mean, rstd, dh, ld[2], dx, dw, db, rows, d, xt, wt, ws, n,
                                                     None))


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), BAD), (dict(d=-1), BAD), (dict(xt=gb.INT8), UNSUP), (dict(wt=gb.F16), UNSUP), (dict(rows=2 ** 31 + 1), UNSUP),
    (dict(dy=None), BAD), (dict(h=None), BAD), (dict(w=None), BAD), (dict(mean=None), BAD), (dict(rstd=None), BAD), (dict(dx=None), BAD),
    (dict(dw=None), BAD), (dict(dw=17), BAD), (dict(db=17), BAD), (dict(ws=18), BAD), (dict(dx=16), BAD), (dict(dx=17), BAD),
    (dict(rstd=18), BAD), (dict(mean=18), BAD), (dict(ld=(7, 8, 8)), BAD), (dict(ld=(8, 7, 8)), BAD), (dict(dh=16, ld=(8, 8, 7)), BAD),
    (dict(dh=17), BAD), (dict(d=0, dw=None), gb.OK),
])
def test_backward_refusals(kw, want):
    assert back(**kw) == want


def test_backward_workspace():
    lib, n, m = gb.load(), ctypes.c_size_t(), ctypes.c_size_t()
    f = lib.gemm_bt_layer_norm_backward_workspace
    assert f(4, 8, None) == BAD and f(-1, 8, ctypes.byref(n)) == BAD and f(2, (1 << 26) + 1, ctypes.byref(n)) == UNSUP and n.value == 0
    for rows, d in ((1, 1), (1000, 2050), (512, 8193), (100000, 64), (3, 100000), (8192, 4096)):
        assert f(rows, d, ctypes.byref(n)) == gb.OK
        assert lib.gemm_bt_rms_norm_backward_workspace(rows, d, ctypes.byref(m)) == gb.OK
        assert n.value == 2 * m.value  # two sums over rows where the other norm has one


def test_wrappers_check_before_the_library():
    x, w, m = torch.zeros(2, 16), torch.ones(16), torch.zeros(2)
    for call in (lambda: gb.add_layer_norm(x, w, w), lambda: gb.add_layer_norm_backward(x, x, w, m, m)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_wrapper_refusals(gpu):
    x, w, m = torch.zeros(2, 16, device="cuda").bfloat16(), torch.ones(16, device="cuda"), torch.zeros(2, device="cuda")
    for error, call in ((ValueError, lambda: gpu.add_layer_norm(x, w[:8])), (ValueError, lambda: gpu.add_layer_norm(x, w, w[:8])),
                        (TypeError, lambda: gpu.add_layer_norm(x, w, w.bfloat16())), (TypeError, lambda: gpu.add_layer_norm(x, w.half())),
                        (TypeError, lambda: gpu.add_layer_norm(x.to(torch.int8), w)),
                        (TypeError, lambda: gpu.add_layer_norm(x, w, out_dtype=torch.float8_e5m2)),
                        (ValueError, lambda: gpu.add_layer_norm(x, w, residual=x[:1])),
                        (ValueError, lambda: gpu.add_layer_norm(x, w, h_out=x)), (ValueError, lambda: gpu.add_layer_norm(x[0, 0], w)),
                        (ValueError, lambda: gpu.add_layer_norm(x, w.cpu())),
                        (ValueError, lambda: gpu.add_layer_norm_backward(x, x.float(), w, m, m)),
                        (ValueError, lambda: gpu.add_layer_norm_backward(x, x, w, m[:1], m)),
                        (ValueError, lambda: gpu.add_layer_norm_backward(x, x, w, m, m.double())),
                        (ValueError, lambda: gpu.add_layer_norm_backward(x, x, w, m, m, dh=x[:1]))):
        with pytest.raises(error):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [3, 64, 511, 1000, 4096, 6001, 16384, 20000])
def test_codes_are_those_of_64_bits(gpu, d):
    """The codes of the exact rows, but for values within fp32's rounding of a step's edge: y / scale is rounded once to
    fp32, 2^-24 of it, and what 64 bits leave out, d 2^-53 and less of the terms of y, is within 2^-36 of them for
    d < 2^17.  (x and the residual are multiples of 2^-6 below 2^6, so their sum is exact in fp32.)"""
    for k, (dt, wt, res, bias) in enumerate(itertools.product(DT, ("own", "f32"), (0, 1), (0, 1))):
        rows, seed = (5, 600)[k % 2], 77 * d + k
        say("layer norm codes", rows, d, dt, wt, res, bias, "seed", seed)
        grid = lambda s, std: ((randn(s, rows, d, std=std) * 64).round() / 64).clamp(-63, 63).to(DT[dt])
        x, r = grid(seed, 2.0), grid(seed + 1, 3.0) if res else None
        w_dt = DT[dt] if wt == "own" else torch.float32
        w = (1 + randn(seed + 2, d, std=0.3)).to(w_dt)
        b = randn(seed + 3, d, std=0.5).to(w_dt) if bias else None
        for out in ("e4m3", "i8"):
            got = gpu.add_layer_norm(x.cuda(), w.cuda(), None if b is None else b.cuda(), residual=None if r is None else r.cuda(),
                                     eps=EPS, out_dtype=EIGHT[out])
            y = norm64(x, r, w, b)[0][3]
            terms = y.abs() + (0 if b is None else 2 * b.double().abs())
            scale = torch.clamp(y.abs().amax(-1) / QMAX[out], min=2.0 ** -100)
            assert bool(((got.scale.cpu().double() - scale).abs() <= u * scale + 2.0 ** -36 * terms.amax(-1) / QMAX[out]).all())
            v, t = y / scale[:, None], 2.0 ** -36 * terms / scale[:, None]
            top = (v.abs() + t) * (1 + 1e-6)
            half = torch.full_like(v, 0.5) if out == "i8" else torch.exp2(torch.floor(torch.log2(top.clamp_min(2.0 ** -6))) - 4)
            off = (got.y.float().double().cpu() - v).abs()
            assert bool((off <= half + 2 * u * v.abs() + 2 * t).all()), (dt, wt, res, bias, out, float((off - half).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("d", [6, 40, 2048, 6000, 20000])
def test_codes_of_extremes(gpu, d, dt):
    """Squares outside fp32's range, centred values outside it, and rows of one value (y is 0, or b)."""
    big = torch.finfo(DT[dt]).max
    x = randn(3, 4, d)
    x[0] = big
    x[0, ::2] = -big
    x[1] *= 2.0 ** -20
    x[2] = big
    x[2, 0] = -big
    x[3] = 2.5
    x = x.to(DT[dt])
    w, b = torch.ones(d), randn(4, d, std=0.5)
    for qt, bias in itertools.product(EIGHT, (None, b)):
        say("layer norm codes of extremes", d, dt, qt, bias is not None)
        got = gpu.add_layer_norm(x.cuda(), w.cuda(), None if bias is None else b.cuda(), eps=EPS, out_dtype=EIGHT[qt])
        (_, _, _, y64), (_, _, t_y) = norm64(x, None, w, bias)
        check_codes(got.y, got.scale, y64, t_y, qt, (d, dt, qt))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [1000, 4096, 20000])
def test_codes_are_rounded_once(gpu, d):
    """Four million values: the codes are those of y / scale unless it lies within 64 bits' errors of a step's edge: d 2^-53
    of the terms of y, which are below 4 times the row's largest value, and so below 2^-36 448 in units of the scale.  A
    rounding to fp32 before the codes would change 1 in 3e6 of them, one of y as many again."""
    rows = 4_000_000 // d
    say("layer norm codes, once", rows, d)
    x, w, b = randn(d, rows, d, std=2.0), 1 + randn(d + 1, d, std=0.3), randn(d + 2, d, std=0.5)
    y = norm64(x, None, w, b)[0][3]
    v = y * QMAX["e4m3"] / y.abs().amax(-1, keepdim=True)
    got = gpu.add_layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS, out_dtype=EIGHT["e4m3"]).y.float().double().cpu()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    t = v / step
    edge = (t - t.floor() - 0.5).abs()
    bad = (got != torch.round(t) * step) & (edge * step > 2.0 ** -36 * 448)
    assert not bool(bad.any()), (d, int(bad.sum()))
