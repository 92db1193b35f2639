"""Group norm with an activation on the GPU against its 64-bit form
(dense_ref), element by element within the bounds derived there."""
import dense_ref as ref
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


@pytest.fixture(scope="module")
def mqc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import im2col_gemm_b200
    return im2col_gemm_b200


def make(n, c, h, w, dtype, seed=0, offset=0.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    last = lambda t: t.to(dtype).permute(0, 3, 1, 2)  # noqa: E731
    return dict(x=last(r(n, h, w, c) + offset * r(c)), g=last(r(n, h, w, c)), gamma=1 + 0.2 * r(c), beta=0.3 * r(c))


def near(got, want, bound, what):
    bound = bound + ref.half_step(want.abs() + bound, got.dtype)
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"off {err[bad][0].item():.3g}, allowed {bound[bad][0].item():.3g}")


def check_fwd(mqc, t, groups, act, eps=EPS):
    y, mean, rstd = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], eps, act)
    r = ref.GroupNorm(t["x"], groups, t["gamma"], t["beta"], eps, act)
    near(mean, r.mean, r.e_mean, "mean")
    near(rstd, r.rstd, r.e_rstd, "rstd")
    near(y, *r.forward(), "y")
    return y, mean, rstd


def check_bwd(mqc, t, groups, act):
    r = ref.GroupNorm(t["x"], groups, None, None, EPS, 0)
    mean, rstd = r.mean.float(), r.rstd.float()
    got = mqc.group_norm_bwd(t["g"], t["x"], groups, mean, rstd, t["gamma"], t["beta"], act)
    want, bounds = ref.GroupNorm(t["x"], groups, t["gamma"], t["beta"], EPS, act, mean, rstd).backward(t["g"])
    for o, v, e, what in zip(got, want, bounds, ("gx", "ggamma", "gbeta")):
        near(o, v, e, what)
    return got


SHAPES = [  # (N, C, H, W, groups)
    (1, 1, 1, 1, 1), (1, 8, 1, 1, 2), (3, 7, 1, 1, 7), (2, 30, 5, 7, 3), (1, 256, 14, 14, 32), (2, 64, 9, 8, 8),
    (2, 320, 20, 20, 32), (1, 33, 17, 3, 11), (5, 12, 64, 1, 4), (1, 16, 1, 1000, 1), (4, 2048, 3, 3, 32),
    (2, 4104, 4, 4, 8), (1, 16, 200, 200, 4), (40, 24, 6, 6, 24), (1, 514, 31, 33, 2), (300, 16, 3, 3, 4),
    (2, 1024, 40, 40, 32), (1, 96, 160, 160, 32), (1, 4096, 9, 9, 1), (3, 2051, 7, 5, 1), (4, 64, 160, 160, 16),
    (1, 924, 53, 88, 4), (6, 34, 64, 64, 2),
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(mqc, shape, dtype):
    *dims, groups = shape
    check_fwd(mqc, make(*dims, dtype, seed=sum(dims)), groups, 2)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(mqc, shape, dtype):
    *dims, groups = shape
    check_bwd(mqc, make(*dims, dtype, seed=sum(dims) + 1), groups, 2)


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("params", ["both", "gamma", "none"])
def test_activations_and_parameters(mqc, act, params):
    t = make(3, 48, 10, 9, F32, seed=act)
    if params != "both":
        t["beta"] = None
    if params == "none":
        t["gamma"] = None
    check_fwd(mqc, t, 6, act)
    check_bwd(mqc, t, 6, act)


@pytest.mark.parametrize("shape", [(2, 16, 8, 8, 4), (1, 64, 60, 60, 8), (1, 16, 200, 200, 4)])
def test_large_common_offset(mqc, shape):
    """Mean 1000, deviation 1: a variance from the mean of squares would be off
    by 1000^2 U = 6%, outside these bounds at the first two shapes."""
    *dims, groups = shape
    t = make(*dims, F32, offset=0.0)
    t["x"] = t["x"] + 1000.0
    y, mean, rstd = check_fwd(mqc, t, groups, 0)
    r = ref.GroupNorm(t["x"], groups, None, None, EPS, 0)
    assert ((rstd.double() - r.rstd).abs() / r.rstd).max() < 1e-3


def test_constant_and_outlier_groups(mqc):
    t = make(1, 16, 9, 9, F32, offset=0.0)
    x = t["x"].clone(memory_format=torch.channels_last)
    x[:, :4] = 3.25                         # no spread at all: y = act(beta)
    x[0, 4, 0, 0] = 30000.0                 # the first element far from the others
    t["x"] = x
    y, mean, rstd = check_fwd(mqc, t, 4, 2)
    assert (mean[0, 0] == 3.25).all() and torch.allclose(rstd[0, 0], torch.tensor(EPS, device="cuda").rsqrt())
    check_bwd(mqc, t, 4, 2)


def test_non_finite_values_stay_in_their_group(mqc):
    t = make(2, 16, 6, 6, BF16)
    y0, m0, s0 = mqc.group_norm_fwd(t["x"], 4, t["gamma"], t["beta"], EPS, 1)
    x = t["x"].clone(memory_format=torch.channels_last)
    x[1, 5, 2, 3] = float("inf")
    x[0, 15, 0, 0] = float("nan")
    y1, m1, s1 = mqc.group_norm_fwd(x, 4, t["gamma"], t["beta"], EPS, 1)
    hit = torch.zeros(2, 16, dtype=torch.bool)
    hit[1, 4:8] = hit[0, 12:16] = True
    assert torch.equal(y0.permute(0, 1, 2, 3)[~hit], y1[~hit]) and torch.isnan(y1[hit]).all()


def strided(t, gap_c, gap_n):
    """The same values with gaps after every pixel and image, NaN in the gaps."""
    n, c, h, w = t.shape
    whole = torch.full((n, h * w * (c + gap_c) + gap_n), float("nan"), dtype=t.dtype, device=t.device)
    view = torch.as_strided(whole, (n, c, h, w), (whole.shape[1], 1, w * (c + gap_c), c + gap_c))
    view.copy_(t)
    return view, whole


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gap_c,gap_n", [(8, 16), (3, 0), (0, 5), (4, 4)])
@pytest.mark.parametrize("shape", [(3, 16, 5, 6, 4), (1, 96, 160, 160, 32)])
def test_strides_and_untouched_gaps(mqc, shape, gap_c, gap_n, dtype):
    """Gaps between pixels and images: the bounds hold, and the gaps of the
    outputs stay as they were."""
    *dims, groups = shape
    t = make(*dims, dtype, seed=gap_c)
    views = {k: strided(t[k], gap_c, gap_n)[0] for k in ("x", "g")}
    t = {**t, **views}
    for bwd in (False, True):
        out, whole = strided(torch.zeros_like(t["x"]), gap_c, gap_n)
        whole.fill_(5.0)
        r = ref.GroupNorm(t["x"], groups, t["gamma"], t["beta"], EPS, 2)
        if bwd:
            mean, rstd = r.mean.float(), r.rstd.float()
            mqc.group_norm_bwd(t["g"], t["x"], groups, mean, rstd, t["gamma"], t["beta"], 2, out=out)
            want, e = ref.GroupNorm(t["x"], groups, t["gamma"], t["beta"], EPS, 2, mean, rstd).backward(t["g"])
            near(out, want[0], e[0], "gx")
        else:
            mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 2, out=out)
            near(out, *r.forward(), "y")
        out.fill_(5.0)
        assert (whole == 5.0).all()


@pytest.mark.parametrize("shape", [(3, 16, 5, 6, 4), (4, 64, 160, 160, 16)])
def test_interleaved_images(mqc, shape):
    """[H][W][N][C] tensors: the images' pixels alternate in memory."""
    n, c, h, w, groups = shape
    t = make(n, c, h, w, BF16)
    mix = lambda v: v.permute(2, 3, 0, 1).contiguous().permute(2, 3, 0, 1)  # noqa: E731
    y0, mean, rstd = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 2)
    x = mix(t["x"])
    y1 = mqc.group_norm_fwd(x, groups, t["gamma"], t["beta"], EPS, 2, out=torch.empty_like(x))[0]
    assert x.stride()[0] == c and torch.equal(y0, y1)
    a = mqc.group_norm_bwd(t["g"], t["x"], groups, mean, rstd, t["gamma"], t["beta"], 2)
    b = mqc.group_norm_bwd(mix(t["g"]), x, groups, mean, rstd, t["gamma"], t["beta"], 2, out=torch.empty_like(x))
    for u, v in zip(a, b):
        assert torch.equal(u, v)


@pytest.mark.parametrize("shape", [(2, 32, 8, 8, 4), (1, 96, 160, 160, 32), (4, 64, 160, 160, 16)])
def test_in_place(mqc, shape):
    *dims, groups = shape
    t = make(*dims, BF16)
    y, mean, rstd = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 2)
    x = t["x"].clone(memory_format=torch.channels_last)
    assert torch.equal(mqc.group_norm_fwd(x, groups, t["gamma"], t["beta"], EPS, 2, out=x)[0], y)
    want = mqc.group_norm_bwd(t["g"], t["x"], groups, mean, rstd, t["gamma"], t["beta"], 2)
    for name in ("g", "x"):
        c = {k: t[k].clone(memory_format=torch.channels_last) for k in ("g", "x")}
        got = mqc.group_norm_bwd(c["g"], c["x"], groups, mean, rstd, t["gamma"], t["beta"], 2, out=c[name])
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_empty_batch(mqc):
    x = torch.empty(0, 16, 4, 4, dtype=BF16, device="cuda").to(memory_format=torch.channels_last)
    y, mean, rstd = mqc.group_norm_fwd(x, 4)
    assert y.shape == x.shape and mean.shape == (0, 4)
    gx, ggamma, gbeta = mqc.group_norm_bwd(x, x, 4, mean, rstd)
    assert gx.shape == x.shape and not ggamma.any() and not gbeta.any()


@pytest.mark.parametrize("shape", [(1, 64, 14, 14, 8), (2, 96, 100, 90, 32), (130, 40, 14, 14, 8),
                                   (4, 64, 160, 160, 16), (3, 602, 60, 17, 2)])
def test_same_bits_each_time(mqc, shape):
    *dims, groups = shape
    t = make(*dims, BF16)
    runs = []
    for _ in range(3):
        f = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 2)
        runs.append(f + mqc.group_norm_bwd(t["g"], t["x"], groups, f[1], f[2], t["gamma"], t["beta"], 2))
    for r in runs[1:]:
        for a, b in zip(r, runs[0]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(2, 24, 7, 9, 4), (1, 96, 150, 150, 8)])
def test_gradient_against_differences(mqc, shape):
    """(L(x + hd) - L(x - hd)) / 2h for L = sum(g y), y in fp32: the cut-off is
    of order h^2, the roundings of y leave sum|g y| U / h."""
    *dims, groups = shape
    t = make(*dims, F32, seed=9)
    n, c, hh, w = dims
    gen = torch.Generator(device="cuda").manual_seed(1)
    d = torch.randn(n, hh, w, c, generator=gen, device="cuda").permute(0, 3, 1, 2)
    _, mean, rstd = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 2)
    gx, ggamma, gbeta = mqc.group_norm_bwd(t["g"], t["x"], groups, mean, rstd, t["gamma"], t["beta"], 2)
    h = 1e-2
    loss = lambda x, ga, be: (mqc.group_norm_fwd(x, groups, ga, be, EPS, 2)[0].double() * t["g"].double()).sum()  # noqa: E731
    dg, db = torch.randn(c, generator=gen, device="cuda"), torch.randn(c, generator=gen, device="cuda")
    cases = [((d, 0 * dg, 0 * db), (gx.double() * d.double()).sum(), (gx.double() * d.double()).square().sum().sqrt()),
             ((0 * d, dg, 0 * db), (ggamma.double() * dg.double()).sum(), ggamma.double().norm()),
             ((0 * d, 0 * dg, db), (gbeta.double() * db.double()).sum(), gbeta.double().norm())]
    for (a, b, e), want, size in cases:
        up = loss(t["x"] + h * a, t["gamma"] + h * b, t["beta"] + h * e)
        down = loss(t["x"] - h * a, t["gamma"] - h * b, t["beta"] - h * e)
        got = (up - down) / (2 * h)
        # h^2 / 6 times a third derivative of order one for each element, as a
        # random sum, and the roundings of y as another
        rounding = (t["g"].double().square().sum().sqrt() * 8 * ref.U * 4) / h
        assert (got - want).abs() <= 20 * h * h * (size + t["g"].double().norm()) + 8 * rounding


def test_captured_and_replayed_on_another_stream(mqc):
    shapes = [(1, 64, 14, 14, 8), (2, 96, 100, 90, 32), (3, 33, 20, 20, 11)]
    ts = [make(*s[:4], BF16, seed=i) for i, s in enumerate(shapes)]

    def run(t, groups):
        f = mqc.group_norm_fwd(t["x"], groups, t["gamma"], t["beta"], EPS, 2)
        return f + mqc.group_norm_bwd(t["g"], t["x"], groups, f[1], f[2], t["gamma"], t["beta"], 2)
    want = [run(t, s[4]) for t, s in zip(ts, shapes)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = [run(t, s[4]) for t, s in zip(ts, shapes)]
    side = torch.cuda.Stream()
    for _ in range(2):
        for outs in got:
            for o in outs:
                o.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_workspace_and_outputs_between_guard_bands(mqc):
    for (n, c, h, w, groups) in [(1, 7, 3, 3, 7), (2, 96, 100, 90, 32), (3, 40, 30, 30, 8)]:
        t = make(n, c, h, w, BF16)
        xd = mqc.T4(n, c, h, w, *t["x"].stride())
        sizes = dict(y=n * c * h * w * 2, mean=n * groups * 4, rstd=n * groups * 4, gg=c * 4, gb=c * 4,
                     ws=max(mqc.mqc_group_norm_fwd_workspace_bytes(xd, xd, mqc.BF16, groups),
                                mqc.mqc_group_norm_bwd_workspace_bytes(xd, xd, xd, mqc.BF16, groups), 1))
        bufs = {k: torch.full((v + 8192,), 0x5A, dtype=torch.uint8, device="cuda") for k, v in sizes.items()}
        at = {k: v.data_ptr() + 4096 for k, v in bufs.items()}
        p = lambda v: v.data_ptr()  # noqa: E731
        for bwd in (False, True):
            if bwd:
                mqc.check(mqc.mqc_group_norm_bwd(p(t["g"]), mqc.T4(n, c, h, w, *t["g"].stride()), p(t["x"]), xd,
                                                 mqc.BF16, p(t["gamma"]), p(t["beta"]), at["mean"], at["rstd"], groups,
                                                 2, at["y"], xd, at["gg"], at["gb"], at["ws"], sizes["ws"], None))
            else:
                mqc.check(mqc.mqc_group_norm_fwd(p(t["x"]), xd, mqc.BF16, p(t["gamma"]), p(t["beta"]), groups, EPS, 2,
                                                 at["y"], xd, at["mean"], at["rstd"], at["ws"], sizes["ws"], None))
            torch.cuda.synchronize()
            for k, v in sizes.items():
                assert (bufs[k][:4096] == 0x5A).all() and (bufs[k][4096 + v:] == 0x5A).all(), k


def test_helper_refusals(mqc):
    t = make(2, 16, 4, 4, BF16)
    with pytest.raises(mqc.MqcError, match="channels last"):
        mqc.group_norm_fwd(t["x"].contiguous(), 4)
    with pytest.raises(mqc.MqcError, match="divide"):
        mqc.group_norm_fwd(t["x"], 5)
    for call in (lambda: mqc.group_norm_fwd(t["x"], 4, t["gamma"][:8]), lambda: mqc.group_norm_fwd(t["x"][0], 4),
                 lambda: mqc.group_norm_fwd(t["x"], 4, t["gamma"].to(BF16)),
                 lambda: mqc.group_norm_fwd(t["x"], 4, out=t["x"][:1])):
        with pytest.raises(ValueError):
            call()


# Large images, whose statistics are joined from the sums of many slabs: 256
# groups of one channel side by side, one group, groups of two, eight channels.
SLABS = [(1, 256, 180, 180, 256), (1, 64, 300, 300, 1), (2, 512, 60, 60, 256), (1, 8, 250, 250, 8)]


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("shape", SLABS)
def test_statistics_of_many_slabs(mqc, shape, dtype):
    *dims, groups = shape
    t = make(*dims, dtype, seed=groups)
    check_fwd(mqc, t, groups, 2)
    check_bwd(mqc, t, groups, 2)


@pytest.mark.parametrize("shape", SLABS)
def test_offsets_of_many_slabs(mqc, shape):
    """A mean of 1000 that drifts by 8 over the image: slabs with means of
    their own, whose spread belongs to the variance."""
    *dims, groups = shape
    t = make(*dims, F32, offset=0.0)
    drift = torch.linspace(996.0, 1004.0, dims[2], device="cuda").view(1, 1, -1, 1)
    t["x"] = (t["x"] + drift).contiguous(memory_format=torch.channels_last)
    check_fwd(mqc, t, groups, 0)


@pytest.mark.parametrize("where", [(0, 0), (90, 17)])
def test_infinity_in_a_slab(mqc, where):
    """One infinity, in the first slab or a later one: its group's mean is
    infinite, its outputs NaN, and the other groups keep their bits."""
    t = make(1, 64, 180, 180, F32)
    clean = mqc.group_norm_fwd(t["x"], 32, t["gamma"], t["beta"], EPS, 2)
    x = t["x"].clone(memory_format=torch.channels_last)
    x[0, 4, where[0], where[1]] = float("inf")
    y, mean, rstd = mqc.group_norm_fwd(x, 32, t["gamma"], t["beta"], EPS, 2)
    others = [g for g in range(32) if g != 2]
    assert mean[0, 2] == float("inf") and torch.isnan(rstd[0, 2]) and torch.isnan(y[0, 4:6]).all()
    assert torch.equal(mean[0, others], clean[1][0, others]) and torch.equal(rstd[0, others], clean[2][0, others])
    assert torch.equal(y[0, 6:], clean[0][0, 6:]) and torch.equal(y[0, :4], clean[0][0, :4])
