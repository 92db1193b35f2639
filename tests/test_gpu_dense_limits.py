"""Group norm where its values, sums or statistics run to their limits, against
the 64-bit form within bounds that stay below the values (dense_bounds)."""
import dense_bounds as tight
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def mqc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import im2col_gemm_b200
    return im2col_gemm_b200


def make(n, c, h, w, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    last = lambda t: t.to(dtype).permute(0, 3, 1, 2)  # noqa: E731
    return dict(x=last(r(n, h, w, c) + 0.5 * r(c)), g=last(r(n, h, w, c)), gamma=1 + 0.2 * r(c), beta=0.3 * r(c))


def within(got, want, bound, what):
    bad = tight.outside(got, want, bound, got.dtype)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item():.6g} for {want[bad][0].item():.6g}, allowed {bound[bad][0].item():.3g}")


def check_bwd(mqc, t, groups, act, run=None):
    r = tight.GroupNorm(t["x"], groups, None, None, EPS, 0)
    mean, rstd = r.mean.float(), r.rstd.float()
    got = mqc.group_norm_bwd(t["g"], t["x"], groups, mean, rstd, t["gamma"], t["beta"], act)
    want, bounds = tight.GroupNorm(t["x"], groups, t["gamma"], t["beta"], EPS, act, mean, rstd, run).backward(t["g"])
    for o, v, e, what in zip(got, want, bounds, ("gx", "ggamma", "gbeta")):
        within(o, v, e, what)


# On chip, in two passes, and with one channel a vector.
FAR = [(2, 32, 8, 8, 4), (1, 32, 400, 400, 4), (2, 35, 9, 9, 5)]
LOW = [-44.0, -62.0, -70.0, -86.0, -104.0, -200.0, -1e4, -1e10, -1e20, -1e30]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", FAR)
def test_silu_far_below_zero_forward(mqc, shape, dtype):
    """SiLU goes to 0 towards -infinity (a beta as a mask), is NaN at it, and a
    channel knows nothing of its neighbours' values."""
    *dims, groups = shape
    t = make(*dims, dtype, seed=1)
    for i, low in enumerate(LOW):
        t["beta"][2 * i + 1] = low          # beside an ordinary channel
    t["beta"][24:31] = torch.tensor([-1e30, -1e20, NAN, 0.5, -INF, 0.25, 60.0])
    y = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 2)[0]
    within(y, *tight.GroupNorm(t["x"], groups, t["gamma"], t["beta"], EPS, 2).forward(), "y")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", FAR)
def test_silu_far_below_zero_backward(mqc, shape, dtype):
    """The slope goes to 0 too: a masked channel leaves its group's gradient alone."""
    *dims, groups = shape
    t = make(*dims, dtype, seed=2)
    for i, low in enumerate(LOW):
        t["beta"][2 * i + 1] = low
    t["beta"][24:27] = torch.tensor([-1e30, -1e20, 60.0])
    check_bwd(mqc, t, groups, 2)


# One CTA, a cluster of four (on chip: no workspace), two passes.
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("shape,dtype", [((2, 128, 6, 6, 32), BF16), ((8, 128, 80, 80, 32), BF16),
                                         ((1, 64, 180, 180, 32), F32)])
def test_an_infinity_leaves_an_infinite_mean(mqc, shape, dtype, value, where):
    """In whichever part of the image it lies; the outputs of its group are
    NaN, and the other groups keep their bits."""
    n, c, h, w, groups = shape
    t = make(n, c, h, w, dtype, seed=3)
    xd = mqc.T4(n, c, h, w, *t["x"].stride())
    code = mqc.F32 if dtype == F32 else mqc.BF16
    assert (mqc.mqc_group_norm_fwd_workspace_bytes(xd, xd, code, groups) == 0) == (h != 180)
    clean = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 2)
    x = t["x"].clone(memory_format=torch.channels_last)
    per = c // groups
    x[n - 1, 2 * per, round(where * (h - 1)), round(where * (w - 1))] = value
    y, mean, rstd = mqc.group_norm_fwd(x, groups, t["gamma"], t["beta"], EPS, 2)
    hit = torch.zeros(n, groups, dtype=torch.bool)
    hit[n - 1, 2] = True
    assert mean[hit].item() == value and torch.isnan(rstd[hit]).all()
    assert torch.equal(mean[~hit], clean[1][~hit]) and torch.equal(rstd[~hit], clean[2][~hit])
    hit = hit.repeat_interleave(per, 1)
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[0][~hit])
