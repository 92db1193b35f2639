"""The linear layer on the GPU against its 64-bit form (dense_ref), element by
element within the bounds derived there."""
import dense_ref as ref
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def mqc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import im2col_gemm_b200
    return im2col_gemm_b200


def make(m, n, k, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(x=r(m, k).to(dtype), w=(r(n, k) * k ** -0.5).to(dtype), bias=r(n), residual=r(m, n).to(dtype),
                g=r(m, n).to(dtype), z=r(m, n).to(dtype))


def near(got, want, bound, dtype):
    bound = bound + ref.half_step(want.abs() + bound, dtype)
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"off {err[bad][0].item():.3g}, allowed {bound[bad][0].item():.3g}")


def check_fwd(mqc, t, act, bias=True, residual=True, save_z=True):
    b, r = t["bias"] if bias else None, t["residual"] if residual else None
    y, z = mqc.linear_fwd(t["x"], t["w"], b, act, r, save_z=save_z)
    mqc.check(mqc.get_device_status())
    wy, wz, ey, ez = ref.linear_fwd(t["x"], t["w"], b, act, r)
    near(y, wy, ey, y.dtype)
    if save_z:
        near(z, wz, ez, z.dtype)
    else:
        assert z is None
    return y


def check_bwd(mqc, t, act):
    got = mqc.linear_bwd(t["g"], t["x"], t["w"], t["z"], act)
    mqc.check(mqc.get_device_status())
    want, bounds = ref.linear_bwd(t["g"], t["x"], t["w"], t["z"], act)
    for o, v, e in zip(got, want, bounds):
        near(o, v, e, o.dtype)
    return got


SHAPES = [  # (M, N, K)
    (1, 1, 1), (3, 5, 7), (1, 4096, 512), (1, 264, 4104), (2, 130, 64), (15, 129, 72), (16, 256, 1024),
    (17, 33, 8), (48, 640, 2560), (64, 128, 128), (65, 200, 72), (127, 129, 65), (128, 1003, 515), (300, 256, 1000),
    (509, 777, 1003), (2000, 40, 24), (5000, 16, 16), (64, 64, 5000), (700, 512, 64),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(mqc, shape, dtype):
    check_fwd(mqc, make(*shape, dtype, seed=sum(shape)), 2)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(mqc, shape, dtype):
    check_bwd(mqc, make(*shape, dtype, seed=sum(shape) + 1), 2)


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("bias,residual,save_z", [(False, False, False), (True, False, True), (False, True, False)])
@pytest.mark.parametrize("shape", [(5, 72, 40), (200, 136, 96), (1100, 1030, 96)])
def test_epilogue(mqc, shape, act, bias, residual, save_z):
    check_fwd(mqc, make(*shape, BF16, seed=act), act, bias, residual, save_z)


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("shape", [(5, 72, 40), (200, 131, 96), (1100, 264, 1030)])
def test_backward_activations(mqc, shape, act):
    check_bwd(mqc, make(*shape, F16, seed=act), act)


# many tiles a processor, ragged on every side, both kinds of row stride
LARGE = [(4096, 4096, 512), (2500, 3000, 264), (2501, 3001, 515), (8192, 520, 136), (300, 8200, 1024)]


@pytest.mark.parametrize("shape", LARGE)
def test_large_forward(mqc, shape):
    check_fwd(mqc, make(*shape, BF16, seed=sum(shape)), 3)


@pytest.mark.parametrize("shape", LARGE)
def test_large_backward(mqc, shape):
    check_bwd(mqc, make(*shape, BF16, seed=sum(shape)), 3)


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True),
                                  (True, False, True), (False, False, False)])
def test_backward_of_what_is_needed(mqc, need):
    t = make(130, 70, 90, BF16)
    full = mqc.linear_bwd(t["g"], t["x"], t["w"], t["z"], 2)
    got = mqc.linear_bwd(t["g"], t["x"], t["w"], t["z"], 2, *need)
    for a, b, n in zip(got, full, need):
        assert (a is None) == (not n)
        assert a is None or torch.equal(a, b)


def padded(t, extra, fill=float("nan")):
    """The same matrix inside rows of `extra` more elements, and the whole buffer."""
    m, n = t.shape
    whole = torch.full((m + 2, n + extra), fill, dtype=t.dtype, device=t.device)
    view = whole[1:1 + m, :n] if (n + extra) * t.element_size() % 16 == 0 else whole[:m, :n]
    view.copy_(t)
    return view, whole


@pytest.mark.parametrize("shape", [(3, 72, 40), (130, 264, 96), (1500, 1304, 200), (1500, 1301, 200), (2000, 2045, 67)])
@pytest.mark.parametrize("extra", [8, 24, 3])
def test_strides_and_untouched_padding(mqc, shape, extra):
    """Rows with a gap between them (NaN there): inputs give the same bits as
    without it, and outputs leave it as it was."""
    m, n, k = shape
    t = make(m, n, k, BF16, seed=extra)
    y0, _ = mqc.linear_fwd(t["x"], t["w"], t["bias"], 2, t["residual"])
    x, w, r = (padded(t[v], extra)[0] for v in ("x", "w", "residual"))
    out, whole = padded(torch.zeros_like(y0), extra, fill=7.0)
    before = whole.clone()
    y1, _ = mqc.linear_fwd(x, w, t["bias"], 2, r, out=out)
    mqc.check(mqc.get_device_status())
    assert y1 is out and torch.equal(y0, out)
    out.copy_(torch.zeros_like(out))
    assert torch.equal(whole, before)
    full = mqc.linear_bwd(t["g"], t["x"], t["w"], t["z"], 2)
    got = mqc.linear_bwd(padded(t["g"], extra)[0], x, w, padded(t["z"], extra)[0], 2)
    for a, b in zip(got, full):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(1, 64, 64), (33, 72, 136), (1200, 1304, 72)])
def test_residual_in_place(mqc, shape):
    t = make(*shape, F16)
    want, _ = mqc.linear_fwd(t["x"], t["w"], t["bias"], 1, t["residual"])
    y = t["residual"].clone()
    mqc.linear_fwd(t["x"], t["w"], t["bias"], 1, y, out=y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("m", [4, 200, 1400])
def test_non_finite_rows_stay_in_their_rows(mqc, m):
    n, k = 1304, 96
    t = make(m, n, k, BF16)
    y0, _ = mqc.linear_fwd(t["x"], t["w"], t["bias"], 0, t["residual"])
    x = t["x"].clone()
    x[m // 2, 3], x[m - 1, k - 1] = float("inf"), float("nan")
    y1, _ = mqc.linear_fwd(x, t["w"], t["bias"], 0, t["residual"])
    rows = torch.ones(m, dtype=torch.bool)
    rows[m // 2] = rows[m - 1] = False
    assert torch.equal(y0[rows], y1[rows])
    assert torch.isnan(y1[m - 1]).all() and not torch.isfinite(y1[m // 2]).all()


def test_relu_passes_nan_on_and_silu_takes_infinities(mqc):
    x = torch.zeros(2, 8, dtype=BF16, device="cuda")
    w = torch.zeros(8, 8, dtype=BF16, device="cuda")
    bias = torch.tensor([float("nan"), float("inf"), -200.0, 200.0, 0.0, -88.0, -100.0, 1.0], device="cuda")
    y, z = mqc.linear_fwd(x, w, bias, 1, save_z=True)
    assert torch.isnan(y[0, 0]) and y[0, 1] == float("inf") and y[0, 2] == 0 and y[0, 3] == 200
    y, z = mqc.linear_fwd(x, w, bias, 2, save_z=True)
    assert torch.isnan(y[0, 0]) and y[0, 1] == float("inf") and y[0, 2] == 0 and y[0, 3] == 200
    assert abs(y[0, 5].item()) < 1e-35 and z[0, 5] == -88


def test_empty_batch(mqc):
    w = torch.randn(24, 16, device="cuda").to(BF16)
    x, g = torch.empty(0, 16, dtype=BF16, device="cuda"), torch.empty(0, 24, dtype=BF16, device="cuda")
    y, z = mqc.linear_fwd(x, w, None, 2, save_z=True)
    assert y.shape == (0, 24) and z.shape == (0, 24)
    gx, gw, gb = mqc.linear_bwd(g, x, w, g, 2)
    assert gx.shape == (0, 16) and not gw.any() and not gb.any()


@pytest.mark.parametrize("shape", [(1, 4096, 4096), (509, 777, 1003), (4096, 2048, 520)])
def test_same_bits_each_time(mqc, shape):
    t = make(*shape, BF16)
    runs = [(mqc.linear_fwd(t["x"], t["w"], t["bias"], 2, t["residual"], save_z=True),
             mqc.linear_bwd(t["g"], t["x"], t["w"], t["z"], 2)) for _ in range(3)]
    for r in runs[1:]:
        for a, b in zip(r[0] + r[1], runs[0][0] + runs[0][1]):
            assert torch.equal(a, b)


def test_linear_gradient_is_the_difference_quotient(mqc):
    """Without an activation the layer is linear: sum(g (y(x + d) - y(x))) is
    sum(gx d) up to the roundings of y (half a step each) and gx."""
    m, n, k = 96, 200, 136
    t = make(m, n, k, F16)
    d = torch.randn(m, k, device="cuda").to(F16)
    xd = (t["x"].float() + d.float()).to(F16)
    step = xd.double() - t["x"].double()
    y0, y1 = (mqc.linear_fwd(v, t["w"])[0].double() for v in (t["x"], xd))
    gx = mqc.linear_bwd(t["g"], t["x"], t["w"])[0].double()
    g = t["g"].double()
    left, right = (g * (y1 - y0)).sum(), (gx * step).sum()
    allowed = (g.abs() * 2.0 ** -11 * (y0.abs() + y1.abs())).sum() + (gx.abs() * 2.0 ** -11 * step.abs()).sum()
    assert (left - right).abs() <= 1.01 * allowed


def test_captured_and_replayed_on_another_stream(mqc):
    cases = [make(1, 512, 1024, BF16), make(200, 264, 72, BF16), make(1500, 1304, 515, BF16)]
    run = lambda t: (mqc.linear_fwd(t["x"], t["w"], t["bias"], 2, t["residual"], save_z=True)  # noqa: E731
                     + mqc.linear_bwd(t["g"], t["x"], t["w"], t["z"], 2))
    want = [run(t) for t in cases]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = [run(t) for t in cases]
    for _ in range(2):
        for outs in got:
            for o in outs:
                o.fill_(float("nan"))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)
    # new values in the same buffers: the graph computes from what is there
    cases[1]["x"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    for u, v in zip(got[1], run(cases[1])):
        assert torch.equal(u, v)


def test_two_streams_at_once(mqc):
    ts = [make(1200, 1304, 200, BF16, seed=s) for s in range(2)]
    run = lambda t: mqc.linear_bwd(t["g"], t["x"], t["w"], t["z"], 2)  # noqa: E731
    want = [run(t) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(ts[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for a, b in zip(outs, want[i]):
                assert torch.equal(a, b)


def test_buffers_end_where_they_end(mqc):
    """Outputs and workspace between guard bands, sizes that end inside a tile."""
    for m, n, k in [(1, 130, 65), (130, 70, 33), (1300, 1100, 65)]:
        t = make(m, n, k, BF16)
        lin = mqc.Linear(m, n, k, mqc.BF16, 2, k, k, n, n, n, n, k, k)
        sizes = dict(y=m * n * 2, z=m * n * 2, gx=m * k * 2, gw=n * k * 2, gb=n * 4,
                     ws=max(mqc.mqc_linear_fwd_workspace_bytes(lin), mqc.mqc_linear_bwd_workspace_bytes(lin)))
        bufs, views = {}, {}
        for name, size in sizes.items():
            bufs[name] = torch.full((size + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
            views[name] = bufs[name].data_ptr() + 4096
        p = lambda v: v.data_ptr()  # noqa: E731
        mqc.check(mqc.mqc_linear_fwd(lin, p(t["x"]), p(t["w"]), p(t["bias"]), None, views["y"], views["z"], views["ws"],
                                     sizes["ws"], None))
        mqc.check(mqc.mqc_linear_bwd(lin, p(t["g"]), views["z"], p(t["x"]), p(t["w"]), views["gx"], views["gw"],
                                     views["gb"], views["ws"], sizes["ws"], None))
        torch.cuda.synchronize()
        mqc.check(mqc.get_device_status())
        for name, size in sizes.items():
            assert (bufs[name][:4096] == 0x5A).all() and (bufs[name][4096 + size:] == 0x5A).all(), name
        y, z = mqc.linear_fwd(t["x"], t["w"], t["bias"], 2, save_z=True)
        assert torch.equal(bufs["y"][4096:4096 + sizes["y"]].view(BF16).view(m, n), y)
        gw = mqc.linear_bwd(t["g"], t["x"], t["w"], z, 2)[1]
        assert torch.equal(bufs["gw"][4096:4096 + sizes["gw"]].view(BF16).view(n, k), gw)


def test_helper_refusals(mqc):
    t = make(8, 16, 24, BF16)
    bad = [lambda: mqc.linear_fwd(t["x"], t["w"][:, :8]), lambda: mqc.linear_fwd(t["x"], t["w"].to(F16)),
           lambda: mqc.linear_fwd(t["x"], t["w"], t["bias"].to(BF16)), lambda: mqc.linear_fwd(t["x"], t["w"].cpu()),
           lambda: mqc.linear_fwd(t["x"], t["w"], residual=t["residual"][:4]),
           lambda: mqc.linear_fwd(t["x"].t().contiguous().t(), t["w"]), lambda: mqc.linear_fwd(t["x"][0], t["w"]),
           lambda: mqc.linear_bwd(t["g"][:, :8], t["x"], t["w"])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mqc.MqcError):
        mqc.linear_fwd(t["x"].float(), t["w"].float())
    with pytest.raises(mqc.MqcError):       # overlapping rows
        mqc.linear_fwd(t["x"][:1].expand(8, 24), t["w"])


@pytest.mark.parametrize("shape", [(1, 203, 72), (40, 203, 512), (130, 203, 72), (300, 1003, 130), (2000, 2045, 64)])
@pytest.mark.parametrize("strides", [(5, 1, 2), (5, 13, 21), (0, 0, 0), (3, 11, 0)])
def test_rows_that_start_anywhere(mqc, shape, strides):
    """y, z and the residual with row strides of their own, alike modulo 16
    bytes or not: pieces of rows are stored whole where they can be, and
    nothing between the rows is touched."""
    m, n, k = shape
    ldy, ldz, ldr = (n + s for s in strides)
    t = make(m, n, k, F16, seed=n)
    y, z, r = (torch.full((m, ld), 7.0, dtype=F16, device="cuda") for ld in (ldy, ldz, ldr))
    r[:, :n] = t["residual"]
    lin = mqc.Linear(m, n, k, mqc.F16, 2, k, k, ldr, ldy, ldz, n, k, k)
    ws = torch.empty(max(1, mqc.lib.mqc_linear_fwd_workspace_bytes(lin)), dtype=torch.uint8, device="cuda")
    mqc.check(mqc.lib.mqc_linear_fwd(lin, t["x"].data_ptr(), t["w"].data_ptr(), t["bias"].data_ptr(), r.data_ptr(),
                                     y.data_ptr(), z.data_ptr(), ws.data_ptr(), ws.numel(),
                                     torch.cuda.current_stream().cuda_stream))
    mqc.check(mqc.get_device_status())
    wy, wz, ey, ez = ref.linear_fwd(t["x"], t["w"], t["bias"], 2, t["residual"])
    near(y[:, :n], wy, ey, F16)
    near(z[:, :n], wz, ez, F16)
    assert (y[:, n:] == 7).all() and (z[:, n:] == 7).all()
