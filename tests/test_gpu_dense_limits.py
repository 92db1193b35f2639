"""Dense layers where their values, sums or statistics run to their limits, against
the 64-bit form within bounds that stay below the values (dense_bounds)."""
import dense_bounds as tight
import dense_ref as ref
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


def make(n, c, h, w, dtype, seed=0, drift=False):
    return tight.make(n, c, h, w, dtype, seed, "cuda", drift)


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


# z is given exactly: beta where a group has no spread, the bias where x is 0.
Z = {2: (-110.0, 30.0), 3: (-14.0, 9.0)}


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pixels", [1, 40000])
@pytest.mark.parametrize("act", [2, 3])
def test_group_norm_activations_at_given_values(mqc, act, pixels, dtype):
    """act and act' themselves, relative to their values, over all that is not
    yet 0 or z: in groups of equal values z is beta, and where there is one
    pixel gbeta is g act'(beta)."""
    c, side = 4096 if pixels == 1 else 64, int(pixels ** 0.5)
    beta = torch.linspace(*Z[act], c, device="cuda")
    x = torch.full((1, side, side, c), 3.25, dtype=dtype, device="cuda").permute(0, 3, 1, 2)
    y, mean, rstd = mqc.group_norm_fwd(x, c // 8, None, beta, EPS, act)
    assert (mean == 3.25).all()
    z = beta.double().view(1, c, 1, 1).expand(x.shape)
    within(y, ref.act(z, act), tight.act_error(z, act) + U_Y * ref.act(z, act).abs(), "y")
    if pixels == 1:
        g = make(1, c, 1, 1, dtype)["g"]
        got = mqc.group_norm_bwd(g, x, c // 8, mean, rstd, None, beta, act)[2]
        s, gd = ref.slope(beta.double(), act), g.double().view(c)
        within(got, gd * s, gd.abs() * (tight.slope_error(beta.double(), act) + U_Y * s.abs()), "gbeta")


U_Y = 2 * ref.U   # a product's rounding, and the sums' that follow


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,n", [(1, 4096), (40, 2048), (129, 1003), (3000, 4096)])
@pytest.mark.parametrize("act", [2, 3])
def test_linear_activations_at_given_values(mqc, act, m, n, dtype):
    """The same for the linear layer: x = 0 leaves z = bias, and with one token
    gb is g act'(z)."""
    bias = torch.linspace(*Z[act], n, device="cuda")
    x, w = torch.zeros(m, 64, dtype=dtype, device="cuda"), torch.ones(n, 64, dtype=dtype, device="cuda")
    y, z = mqc.linear_fwd(x, w, bias, act, save_z=True)
    mqc.check(mqc.get_device_status())
    assert torch.equal(z, bias.to(dtype).expand(m, n))
    exact = bias.double().expand(m, n)
    within(y, ref.act(exact, act), tight.act_error(exact, act) + U_Y * ref.act(exact, act).abs(), "y")
    if m == 1:
        g = make(1, n, 1, 1, dtype)["g"].reshape(1, n)
        gb = mqc.linear_bwd(g, x, w, z, act)[2]
        zd, gd = z.double().view(n), g.double().view(n)
        s = ref.slope(zd, act)
        within(gb, gd * s, gd.abs() * (tight.slope_error(zd, act) + U_Y * s.abs()), "gb")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", FAR)
def test_gelu_over_its_range(mqc, shape, dtype):
    *dims, groups = shape
    t = make(*dims, dtype, seed=4)
    t["beta"] = torch.linspace(-10.0, 8.0, dims[1], device="cuda")
    y = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 3)[0]
    within(y, *tight.GroupNorm(t["x"], groups, t["gamma"], t["beta"], EPS, 3).forward(), "y")
    check_bwd(mqc, t, groups, 3)


def test_gelu_error_of_ordinary_values(mqc):
    """fp32, standard normal z, as a 2-norm: a rounding of z, of the normal
    distribution and of their product, U / sqrt 3 each on average, and half
    again for the distribution's own evaluation (dense_bounds)."""
    t = make(4, 64, 40, 40, F32, seed=5)
    y, mean, rstd = mqc.group_norm_fwd(t["x"], 8, None, None, EPS, 3)
    z = (t["x"].double() - mean.double().repeat_interleave(8, 1)[..., None, None]) * rstd.double().repeat_interleave(
        8, 1)[..., None, None]
    want = ref.act(z, 3)
    assert ((y.double() - want).norm() / want.norm()).item() < 1.5 * ref.U


def in_passes(mqc, t, groups):
    """Whether the forward pass joins slabs: it needs a workspace then."""
    xd = mqc.T4(*t["x"].shape, *t["x"].stride())
    code = {F32: mqc.F32, F16: mqc.F16}[t["x"].dtype]
    return mqc.mqc_group_norm_fwd_workspace_bytes(xd, xd, code, groups) > 0


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("shape", tight.SLABS)
def test_sums_of_many_slabs(mqc, shape, dtype):
    *dims, groups = shape
    t = make(*dims, dtype, seed=groups)
    assert in_passes(mqc, t, groups) or dims[3] == 200 or dtype == F16   # fewer bytes may stay on chip
    y, mean, rstd = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 2)
    r = tight.GroupNorm(t["x"], groups, t["gamma"], t["beta"], EPS, 2, run=tight.RUN)
    within(mean, r.mean, r.e_mean, "mean")
    within(rstd, r.rstd, r.e_rstd, "rstd")
    within(y, *r.forward(), "y")
    check_bwd(mqc, t, groups, 2, tight.RUN)


@pytest.mark.parametrize("shape", tight.SLABS)
def test_drift_over_many_slabs(mqc, shape):
    *dims, groups = shape
    t = make(*dims, F32, seed=groups, drift=True)
    y, mean, rstd = mqc.group_norm_fwd(t["x"], groups, None, None, EPS, 0)
    r = tight.GroupNorm(t["x"], groups, None, None, EPS, 0, run=tight.RUN)
    within(mean, r.mean, r.e_mean, "mean")
    within(rstd, r.rstd, r.e_rstd, "rstd")
    within(y, *r.forward(), "y")
