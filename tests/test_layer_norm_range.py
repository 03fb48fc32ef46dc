"""The layer norm over fp32's whole range, against 64 bits: rows whose squares, or whose sums, leave it though every entry,
centred value and result lies inside, and the statistics of rows that hold an infinity or a NaN.

The tolerances are those of test_layer_norm.py: powers of two that a row's sums are scaled by round nothing, so the bounds
relative to the sum of magnitudes stand.  Entries stay below 2^126 and above 2^60, so that rstd is a normal fp32 number.
"""
import pytest
import torch

from test_layer_norm import EPS, norm64
from test_layers_gpu import DT, close, gen, randn, say

WIDTHS = [8, 40, 700, 1031, 2048, 4096, 8200, 12003, 20000]  # a wave's rows, a workgroup's, ragged ones, and long ones


def check(gpu, x, r, seed, what):
    d = x.shape[1]
    w, b = 1 + randn(seed + 1, d, std=0.3), randn(seed + 2, d, std=0.5)
    g = lambda t: None if t is None else t.cuda()
    got = gpu.add_layer_norm(x.cuda(), w.cuda(), b.cuda(), residual=g(r), eps=EPS, save_stats=True, out_dtype=torch.float32)
    (_, mean, rstd, y64), (t_mean, t_rstd, t_y) = norm64(x, r, w, b)
    mean = torch.where(torch.isnan(rstd), rstd, mean)  # (a row without a value has no mean either, one infinity in it or two)
    close(got.mean, mean, t_mean, ("mean", what))
    close(got.rstd, rstd, t_rstd, ("rstd", what))
    close(got.y, y64, t_y, ("y", what))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_squares_outside_the_range(gpu, d, dt):
    """Ordinary rows of large entries: what the rounding of their first mean leaves out has a square outside fp32 too."""
    for rows, power, mean in ((6, 62, 0.7), (6, 95, 0.0), (6, 95, 0.7), (5, 110, -3.0), (700, 110, 0.2)):
        seed = d + power
        x = ((randn(seed, rows, d) + mean) * 2.0 ** power).to(DT[dt])
        for r in (None, (randn(seed + 9, rows, d) * 2.0 ** (power - 1)).to(DT[dt])):
            say("layer norm, large rows", rows, d, dt, "2 **", power, "mean", mean, r is not None, "seed", seed)
            check(gpu, x, r, seed, (d, dt, power, mean))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("d", WIDTHS)
def test_statistics_of_rows_without_a_value(gpu, d, dt):
    """An infinity or a NaN makes its row's y, mean and rstd NaN, and no other row's."""
    for rows in (7, 700):
        x = randn(d + rows, rows, d)
        x[0, d // 2] = float("inf")
        x[2, d - 1] = float("nan")
        x[3, 0] = -float("inf")
        x[5, 1], x[5, d - 2] = float("inf"), -float("inf")
        x = x.to(DT[dt])
        say("layer norm, rows without a value", rows, d, dt)
        check(gpu, x, None, d, (d, dt, rows))
        got = gpu.add_layer_norm(x.cuda(), torch.ones(d, device="cuda"), eps=EPS, save_stats=True, out_dtype=torch.float8_e4m3fn)
        bad = torch.zeros(rows, dtype=torch.bool)
        bad[[0, 2, 3, 5]] = True
        for t in (got.mean, got.rstd, got.scale):
            assert torch.equal(torch.isnan(t.cpu()), bad), (d, dt, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_nearly_equal_large_entries(gpu, d, dt):
    """Rows of one large value, and of entries a few steps of their type from it: the squares of what is left are inside the
    range again, or 0, where those of what the first mean's rounding leaves out are not."""
    step = 2.0 ** -8 if dt == "bf16" else 2.0 ** -23
    for rows, power in ((6, 100), (6, 118), (700, 118)):
        seed = d + power
        big = (1 + randn(seed, rows, 1).abs()).clamp(max=1.9).to(DT[dt]).float()
        x = big * (1 + step * torch.randint(0, 3, (rows, d), generator=gen(seed))) * 2.0 ** power
        x[::2] = (big * 2.0 ** power)[::2]
        say("layer norm, nearly equal large entries", rows, d, dt, "2 **", power, "seed", seed)
        check(gpu, x.to(DT[dt]), None, seed, (d, dt, power))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_sums_outside_the_range(gpu, d, dt):
    """Runs of large entries of one sign: what a thread, a wave or a workgroup sums on the way is infinite, or infinities of
    both signs meet, in the first mean's sum or in that of what it leaves."""
    size = (1 + 0.1 * randn(d, 6, d).abs()).clamp(max=1.4) * 2.0 ** 125
    sign = torch.ones(6, d)
    sign[0, d // 2:] = -1          # halves
    sign[1, d // 4:] = -1 / 3      # a quarter against the rest
    sign[2, :] = -1                # one sign alone
    sign[3] = 1 - 2 * (torch.arange(d) // 8 % 2)    # a thread's entries of one sign
    sign[4] = 1 - 2 * (torch.arange(d) // 512 % 2)  # a wave's
    sign[5, d // 2:] = 2.0 ** -60
    for rows in (6, 600):
        x = (size * sign).repeat(rows // 6, 1).to(DT[dt])
        for r in (None, (randn(d + 1, rows, d) * 2.0 ** 120).to(DT[dt])):
            say("layer norm, sums outside the range", rows, d, dt, r is not None)
            check(gpu, x, r, d, (d, dt, rows))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [40, 2048, 4096, 20000])
def test_centred_values_outside_the_range(gpu, d):
    """A finite row whose h - mean is infinite somewhere has no value: y, mean and rstd are NaN, and no other row's."""
    big = torch.finfo(torch.float32).max
    x = randn(d, 4, d)
    x[1], x[1, 3] = big, -big
    x[2], x[2, d - 1] = -big, big
    got = gpu.add_layer_norm(x.cuda(), torch.ones(d, device="cuda"), eps=EPS, save_stats=True)
    bad = torch.tensor([False, True, True, False])
    for t in (got.y.cpu(), got.mean.cpu()[:, None], got.rstd.cpu()[:, None]):
        assert torch.equal(torch.isnan(t), bad[:, None].expand_as(t)), d
