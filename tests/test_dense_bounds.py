"""CPU: the bounds that the GPU tests of many slabs use leave out what a wrong
join of the slabs would give."""
import dense_bounds as tight
import pytest
import torch

F32 = torch.float32


def outside(got, want, bound):
    return tight.outside(got.float(), want, bound, F32).double().mean().item()


@pytest.mark.parametrize("shape", tight.SLABS)
def test_wrong_statistics_fall_outside(shape):
    """A variance without the spread between slabs, one of 1, the first slab's
    statistics, and outputs of nothing but zeros, at an offset of 1000."""
    *dims, groups = shape
    t = tight.make(*dims, F32, drift=True)
    n, c, h, w = dims
    r = tight.GroupNorm(t["x"], groups, None, None, tight.EPS, 0, run=tight.RUN)
    assert outside(r.mean, r.mean, r.e_mean) == 0 and outside(r.rstd, r.rstd, r.e_rstd) == 0
    rows = t["x"].double().view(n, groups, c // groups, h, w)
    parts = rows.var((2, 4), unbiased=False).mean(2)          # within each row of pixels
    first = rows[:, :, :, :max(1, h // 64)]
    for wrong in ((parts + tight.EPS).rsqrt(), torch.ones_like(r.rstd),
                  (first.var((2, 3, 4), unbiased=False) + tight.EPS).rsqrt()):
        assert outside(wrong, r.rstd, r.e_rstd) == 1
    assert outside(first.mean((2, 3, 4)), r.mean, r.e_mean) == 1
    y, bound = r.forward()
    assert outside(torch.zeros_like(y), y, bound) > 0.98      # the others are next to 0
    assert outside(y * 2.5, y, bound) > 0.98                  # as with rstd = 1


@pytest.mark.parametrize("shape,pixels", list(zip(tight.SLABS, tight.SLAB_PIXELS)))
def test_wrong_sums_fall_outside(shape, pixels):
    """The parameters' gradients: nothing, or one slab left out or taken twice."""
    *dims, groups = shape
    t = tight.make(*dims, F32)
    args = (groups, t["gamma"], t["beta"], tight.EPS, 2)
    r = tight.GroupNorm(t["x"], *args, run=tight.RUN)
    mean, rstd = r.mean.float(), r.rstd.float()
    (gx, *sums), (e_gx, *bounds) = tight.GroupNorm(t["x"], *args, mean, rstd, tight.RUN).backward(t["g"])
    g = t["g"].clone()
    g.permute(0, 2, 3, 1).view(dims[0], dims[2] * dims[3], dims[1])[0, pixels:] = 0
    g[1:] = 0
    slab = tight.GroupNorm(t["x"], *args, mean, rstd, tight.RUN).backward(g)[0][1:]
    for want, bound, part in zip(sums, bounds, slab):
        assert outside(want, want, bound) == 0
        for wrong in (torch.zeros_like(want), want - part, want + part):
            assert outside(wrong, want, bound) >= 0.85
    assert outside(torch.zeros_like(gx), gx, e_gx) > 0.98
