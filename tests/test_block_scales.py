"""block_linear takes scales of blocks in every layout: strides past what the kernels take, and rows past them."""
import pytest
import torch

from dense_tiled_gemm_amd.layers import _block_scale

F8 = torch.float8_e4m3fn
MANY = 1 << 26


@pytest.mark.parametrize("shape,strides", [
    ((5, 3), (1, 5)), ((5, 3), (3, 1)), ((5, 3), (0, 1)), ((5, 3), (1 << 21, 1)), ((5, 3), (1, 1 << 27)), ((5, 3), (1 << 21, 1 << 27)),
    ((1, 8), (1 << 21, 1)), ((1, 8), (1, 1 << 27)), ((4, 1), (1, 1 << 26)), ((4, 1), (1 << 21, 1)), ((1, 1), (1 << 21, 1 << 27)),
    ((MANY, 1), (1, MANY)), ((MANY, 2), (1, MANY)), ((MANY + 5, 2), (2, 1)), ((0, 3), (1, 0)), ((3, 0), (1, 3)),
])
def test_strides_are_those_the_kernels_take(shape, strides):
    t, row, block = _block_scale(torch.empty_strided(shape, strides, device="meta"), *shape, "x_scale")
    assert t.shape == shape and 0 <= row < 1 << 20 and 0 <= block < 1 << 26
    for n, s, want in zip(shape, t.stride(), (row, block)):
        assert n <= 1 or s == want


@pytest.mark.gpu
def test_far_strides(gpu):
    """The same bits from scales whose rows, or blocks, lie far apart."""
    M, N, K = 3, 300, 384
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randn(n, K, generator=g).to(F8).cuda() for n in (M, N))
    sx, sw = (torch.exp(torch.randn(n, 3, generator=g)).cuda() for n in (M, 3))
    want = gpu.block_linear(x, w, sx, sw)
    wide = torch.zeros(M, (1 << 20) + 7, device="cuda")
    wide[:, 5:8] = sx
    assert torch.equal(gpu.block_linear(x, w, wide[:, 5:8], sw), want)
    for rows in range(1, M):
        assert torch.equal(gpu.block_linear(x[:rows], w, wide[:rows, 5:8], sw), want[:rows])


@pytest.mark.gpu
@pytest.mark.parametrize("K", [16, 144])
def test_more_rows_than_a_block_stride_can_be(gpu, K):
    """2^26 rows and a few, one block along K and two: the scales as quantize_blocks leaves them."""
    M, N = MANY + 37, 4
    print("[case] block linear", M, N, K, flush=True)
    x = torch.randint(0, 100, (M, K), dtype=torch.uint8, device="cuda").view(F8)
    w = torch.randint(0, 100, (N, K), dtype=torch.uint8, device="cuda").view(F8)
    blocks = (K + 127) // 128
    sx, sw = (torch.rand(blocks, M, device="cuda") + 0.5).t(), torch.rand(1, blocks, device="cuda") + 0.5
    y = gpu.block_linear(x, w, sx, sw)
    for rows in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        assert torch.equal(y[rows], gpu.block_linear(x[rows], w, sx[rows].contiguous(), sw))
