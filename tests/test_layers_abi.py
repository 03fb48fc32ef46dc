"""The row operators and the product with an epilogue: what is refused, and what needs no GPU (CPU)."""
import ctypes

import pytest

import dense_tiled_gemm_amd as gb

BAD, UNSUP = gb.ERR_INVALID_VALUE, gb.ERR_UNSUPPORTED
NODEV = (gb.ERR_NO_DEVICE, gb.OK)


def epi(A=16, B=16, C=16, M=4, N=4, K=16, i=gb.BF16, o=gb.BF16, ws=None, ws_bytes=0, **terms):
    from dense_tiled_gemm_amd.layers import Epilogue

    e = Epilogue(**terms)
    return int(gb.load().gemm_bt_epi(A, B, C, M, N, K, i, o, ctypes.byref(e), ws, ws_bytes, None))


@pytest.mark.parametrize("kw,want", [
    (dict(o=gb.INT32), UNSUP),
    (dict(o=gb.FP8_E4M3), UNSUP),
    (dict(i=gb.F32), UNSUP),
    (dict(i=gb.INT8, o=gb.INT32), UNSUP),
    (dict(i=gb.INT8, K=131088), UNSUP),
    (dict(i=gb.FP8_E4M3, K=8), UNSUP),                      # 8-bit rows in whole 16-byte chunks
    (dict(activation=-1), BAD),
    (dict(activation=5), BAD),
    (dict(bias=16, bias_dtype=gb.INT8), BAD),
    (dict(bias=17, bias_dtype=gb.BF16), BAD),               # not aligned to its elements
    (dict(bias=18, bias_dtype=gb.F32), BAD),
    (dict(residual=16, residual_dtype=gb.INT32), BAD),
    (dict(preact=18, preact_dtype=gb.F32), BAD),
    (dict(preact=16, preact_dtype=9), BAD),
    (dict(row_scale=18), BAD),
    (dict(col_scale=2), BAD),
    (dict(bias=None, bias_dtype=77), NODEV),                # the type of an absent term is not read
    (dict(M=-1), BAD),
    (dict(C=None), BAD),
    (dict(C=17), BAD),
    (dict(C=18, o=gb.F32), BAD),
    (dict(C=18, i=gb.INT8), NODEV),                         # 2-byte results of an int8 product
    (dict(A=None), BAD),
    (dict(M=0, A=None, B=None, C=None), gb.OK),
    (dict(N=0, A=None, B=None, C=None), gb.OK),
])
def test_epilogue_refusals(kw, want):
    if isinstance(want, tuple):  # accepted: without a device the call ends at the device check
        import torch

        if torch.cuda.is_available():
            pytest.skip("made-up pointers are for machines without a GPU")
        assert epi(**kw) == gb.ERR_NO_DEVICE
    else:
        assert epi(**kw) == want


def norm(x=16, ldx=8, res=None, ldr=0, w=16, y=16, h=None, scale=None, rstd=None, rows=2, d=8, eps=1e-6, xt=gb.BF16,
         wt=gb.BF16, yt=gb.BF16):
    return int(gb.load().gemm_bt_rms_norm(x, ldx, res, ldr, w, y, h, scale, rstd, rows, d, eps, xt, wt, yt, None))


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), BAD), (dict(d=-1), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(xt=gb.INT8), UNSUP), (dict(wt=gb.F16), UNSUP), (dict(xt=gb.F32, wt=gb.BF16), UNSUP), (dict(yt=gb.FP8_E5M2), UNSUP),
    (dict(yt=gb.INT32), UNSUP), (dict(d=2 ** 31 - 1, ldx=2 ** 31), UNSUP), (dict(rows=2 ** 31 + 1), UNSUP),
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(x=17), BAD), (dict(y=17), BAD),
    (dict(yt=gb.FP8_E4M3), BAD),                             # 8-bit rows without a place for their scales
    (dict(yt=gb.INT8, scale=18), BAD), (dict(rstd=18), BAD), (dict(h=17), BAD),
    (dict(ldx=7), BAD), (dict(res=16, ldr=7), BAD), (dict(res=17, ldr=8), BAD),
    (dict(rows=0, x=None, w=None, y=None), gb.OK), (dict(d=0, x=None, w=None, y=None), gb.OK),
])
def test_norm_refusals(kw, want):
    assert norm(**kw) == want


def test_quantize_refusals():
    q = lambda *a: int(gb.load().gemm_bt_quantize_rows(*a, None))
    assert q(16, 8, 16, 16, -1, 8, gb.BF16, gb.INT8) == BAD
    assert q(16, 8, 16, 16, 2, 8, gb.BF16, gb.FP8_E5M2) == UNSUP
    assert q(16, 8, 16, 16, 2, 8, gb.INT8, gb.INT8) == UNSUP
    assert q(16, 7, 16, 16, 2, 8, gb.BF16, gb.INT8) == BAD
    assert q(16, 8, 16, None, 2, 8, gb.BF16, gb.INT8) == BAD
    assert q(17, 8, 16, 16, 2, 8, gb.BF16, gb.INT8) == BAD
    assert q(None, 8, None, None, 0, 8, gb.BF16, gb.INT8) == gb.OK


def norm_back(dy=16, h=16, w=16, rstd=16, dh=None, dx=32, dw=16, rows=2, d=8, xt=gb.BF16, wt=gb.BF16, ws=16, n=1 << 20,
              ld=(8, 8, 8)):
    return int(gb.load().gemm_bt_rms_norm_backward(dy, ld[0], h, ld[1], w, rstd, dh, ld[2], dx, dw, rows, d, xt, wt, ws, n,
                                                   None))


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), BAD), (dict(d=-1), BAD), (dict(xt=gb.INT8), UNSUP), (dict(wt=gb.F16), UNSUP),
    (dict(dy=None), BAD), (dict(h=None), BAD), (dict(w=None), BAD), (dict(rstd=None), BAD), (dict(dx=None), BAD),
    (dict(dw=None), BAD), (dict(dw=17), BAD), (dict(ws=18), BAD), (dict(dx=16), BAD), (dict(dx=17), BAD), (dict(rstd=18), BAD),
    (dict(ld=(7, 8, 8)), BAD), (dict(ld=(8, 7, 8)), BAD), (dict(dh=16, ld=(8, 8, 7)), BAD), (dict(dh=17), BAD),
    (dict(d=0, dw=None), gb.OK),
])
def test_norm_backward_refusals(kw, want):
    assert norm_back(**kw) == want


def act_back(dy=16, z=16, dz=16, db=16, rows=2, n=8, act=1, t=gb.BF16, zt=gb.BF16, bt=gb.BF16, ws=16, nbytes=1 << 20):
    return int(gb.load().gemm_bt_act_backward(dy, z, dz, db, rows, n, act, t, zt, bt, ws, nbytes, None))


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), BAD), (dict(n=-1), BAD), (dict(act=5), BAD), (dict(act=-1), BAD), (dict(t=gb.INT8), UNSUP),
    (dict(zt=gb.INT8), UNSUP), (dict(bt=gb.INT32), UNSUP), (dict(dy=None), BAD), (dict(z=None), BAD), (dict(ws=None), BAD),
    (dict(ws=18), BAD), (dict(dz=17), BAD), (dict(db=17), BAD), (dict(z=17), BAD),
    (dict(n=0, dy=None), gb.OK), (dict(rows=0, db=None, dy=None), gb.OK), (dict(dz=None, db=None), gb.OK),
])
def test_act_backward_refusals(kw, want):
    assert act_back(**kw) == want


def lin_back(dy=16, x=16, w=16, z=16, dx=16, dw=16, db=16, M=4, N=8, K=8, act=1, t=gb.BF16, zt=gb.BF16, ws=16, nbytes=1 << 30):
    return int(gb.load().gemm_bt_linear_backward(dy, x, w, z, dx, dw, db, M, N, K, act, t, zt, ws, nbytes, None))


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=-1), BAD), (dict(act=9), BAD), (dict(t=gb.F32), UNSUP),
    (dict(M=1 << 30, K=1 << 20), UNSUP), (dict(N=(1 << 21) - 1, K=(1 << 21) - 1), UNSUP),
    (dict(zt=gb.INT8), UNSUP), (dict(N=1 << 21), UNSUP), (dict(K=1 << 21), UNSUP), (dict(dy=None), BAD), (dict(x=None), BAD),
    (dict(w=None), BAD), (dict(z=None), BAD), (dict(dx=17), BAD), (dict(dw=17), BAD), (dict(db=17), BAD), (dict(x=17), BAD),
    (dict(z=17), BAD), (dict(dx=None, dw=None, db=None), gb.OK), (dict(M=0, dw=None, db=None, dy=None), gb.OK),
    (dict(N=0, dx=None, dy=None), gb.OK), (dict(K=0, db=None, dy=None), gb.OK),
])
def test_linear_backward_refusals(kw, want):
    assert lin_back(**kw) == want


def test_linear_backward_workspace():
    lib, n = gb.load(), ctypes.c_size_t()
    size = lambda *a: (lib.gemm_bt_linear_backward_workspace(*a, ctypes.byref(n)), n.value)
    assert lib.gemm_bt_linear_backward_workspace(4, 8, 8, 0, None) == BAD
    assert size(-1, 8, 8, 0) == (BAD, 0) and size(4, 8, 8, 7) == (BAD, 0) and size(4, 1 << 21, 8, 0) == (UNSUP, 0)
    assert size(0, 8, 8, 1) == (gb.OK, 0)
    assert size(4096, 4096, 4096, 3)[1] >= 4096 * 4096 * 2            # dz
    assert size(4096, 4096, 4096, 0)[1] < 4096 * 4096 * 2             # dy is dz
    assert size(100, 9, 8, 0)[1] >= 100 * 16 * 2                      # padded rows of dz
    assert size(100, 8, 9, 0)[1] >= (100 + 8) * 16 * 2                # padded rows of x and w
    # operands past 2 GiB: cut along the sum even where nothing else asks for it
    assert size(1 << 20, 4096, 4096, 0)[1] >= 4 * 4096 * 4096 * 4


def test_epilogue_plans():
    """16-bit products are planned as gemm_bt_ws plans them, but for M <= 16 and few columns; 8-bit ones of few rows stream
    or are cut along K."""
    for i in (gb.BF16, gb.F16):
        p = gb.gemm_bt_plan_epi(1, 4096, 4096, i, i)
        assert (p.kernel, p.bm, p.bn, p.bk, p.split_tiles, p.grid) == (4, 32, 64, 128, 64, 128)
        p = gb.gemm_bt_plan_epi(16, 4096, 1000, i, i)
        assert (p.kernel, p.bm, p.bn, p.split_tiles) == (4, 32, 64, 0)
        assert gb.gemm_bt_plan_epi(1, 4097, 4096, i, i).kernel == 3
        assert gb.gemm_bt_plan_ws(1, 4096, 4096, i, i).kernel == 3
    for i in (gb.BF16, gb.F16):
        p = gb.gemm_bt_plan_epi(1213, 91, 4279, i, i)             # 38 tiles of 64 x 64, 34 steps of 128
        assert (p.bm, p.bn, p.bk, p.split_tiles, p.grid) == (64, 64, 128, 38, 38 * 4)
        assert p.workspace_bytes == 16384 + p.grid * 64 * 64 * 4
        assert gb.gemm_bt_plan_epi(512, 512, 2944, i, i).split_tiles == 0   # 23 steps
        assert gb.gemm_bt_plan_epi(512, 512, 2952, i, i).split_tiles == 64
        assert gb.gemm_bt_plan_epi(1024, 600, 8192, i, i).split_tiles != 160  # more than half the CUs have a tile
    for M, N, K in ((1, 8192, 4096), (17, 4096, 4096), (64, 8192, 8192), (1024, 1024, 16384), (4096, 4096, 4096), (4352, 4096, 4096), (0, 5, 5)):
        for i, o in ((gb.BF16, gb.F32), (gb.F16, gb.F16)):
            assert gb.gemm_bt_plan_epi(M, N, K, i, o).as_dict() == gb.gemm_bt_plan_ws(M, N, K, i, o).as_dict()
    for i in (gb.FP8_E4M3, gb.FP8_E5M2, gb.INT8):
        p = gb.gemm_bt_plan_epi(16, 8192, 8192, i, gb.BF16)
        assert (p.kernel, p.bn, p.bk, p.grid, p.workspace_bytes) == (3, 8, 512, 1024, 0)
        p = gb.gemm_bt_plan_epi(16, 4096, 4096, i, gb.BF16)       # not more than two of its workgroups per CU
        assert (p.kernel, p.bm, p.bk, p.split_tiles, p.grid) == (4, 64, 256, 64, 128)
        p = gb.gemm_bt_plan_epi(64, 8192, 8192, i, gb.BF16)
        assert (p.split_tiles, p.grid, p.workspace_bytes) == (128, 256, 16384 + 256 * 64 * 64 * 4)
        p = gb.gemm_bt_plan_epi(64, 8192, 4080, i, gb.BF16)       # 16 steps: pieces of 8
        assert (p.split_tiles, p.grid) == (128, 256)
        p = gb.gemm_bt_plan_epi(64, 8192, 3840, i, gb.BF16)       # 15 steps: not cut
        assert (p.split_tiles, p.grid, p.variant) == (0, 128, 5)
        p = gb.gemm_bt_plan_epi(4096, 4096, 4096, i, gb.BF16)
        assert (p.bm, p.split_tiles) == (256, 0)
    n = ctypes.c_size_t()
    size = lambda *a: (gb.load().gemm_bt_epi_workspace_size(*a, ctypes.byref(n)), n.value)
    assert size(64, 8192, 8192, gb.INT8, gb.BF16) == (gb.OK, 16384 + 256 * 64 * 64 * 4)
    assert size(64, 8192, 8192, gb.INT8, gb.INT32) == (UNSUP, 0)
    assert size(-1, 8192, 8192, gb.BF16, gb.BF16) == (BAD, 0)
    assert gb.load().gemm_bt_epi_workspace_size(1, 1, 1, gb.BF16, gb.BF16, None) == BAD
    assert gb.load().gemm_bt_plan_epi(1, 1, 1, gb.BF16, gb.INT32, 16, 16, 16, None) == BAD


def test_workspace_sizes():
    lib, n = gb.load(), ctypes.c_size_t()
    for f in (lib.gemm_bt_rms_norm_backward_workspace, lib.gemm_bt_act_backward_workspace):
        assert f(1000, 2050, None) == BAD
        assert f(-1, 8, ctypes.byref(n)) == BAD and n.value == 0
        assert f(2, 2 ** 31 - 1, ctypes.byref(n)) == UNSUP and f(2, (1 << 26) + 1, ctypes.byref(n)) == UNSUP
        assert f(0, 4096, ctypes.byref(n)) == gb.OK and n.value == 0
        for rows, d in ((1, 1), (1000, 2050), (512, 8192), (512, 8193), (512, 4096), (513, 4096), (256, 8), (257, 8), (100000, 64), (1 << 31, 8), (3, 100000), (8192, 4096)):
            assert f(rows, d, ctypes.byref(n)) == gb.OK
            # whole rows of fp32 sums, at most one per row of input; none for the norm of few rows
            threads = 256
            while threads < min(1024, -(-d // 8)):
                threads *= 2
            few = (f is lib.gemm_bt_rms_norm_backward_workspace and rows <= threads and d <= 16384 and rows * d <= 1 << 22)
            assert n.value % (4 * d) == 0 and (0 if few else 1) <= n.value // (4 * d) <= rows
            assert n.value // (4 * d) <= 65535
            assert n.value == 0 if few else n.value > 0


def test_wrappers_check_before_the_library():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 16), torch.zeros(4, 16)
    for call in (lambda: gb.linear(x.bfloat16(), w.bfloat16()), lambda: gb.add_rms_norm(x, torch.ones(16)),
                 lambda: gb.quantize_rows(x), lambda: gb.linear_backward(x, x, w),
                 lambda: gb.add_rms_norm_backward(x, x, x[0], x[:, 0])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(AttributeError):
        gb.no_such_name
