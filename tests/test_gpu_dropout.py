"""Dropout on the GPU: the kept elements are exactly those of the 64-bit form
(numpy's integers), the values within the bounds of dense_ref."""
import dense_ref as ref
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SEED, OFFSET = 0xFEDCBA9876543210, 0x1_0000_0007


@pytest.fixture(scope="module")
def mqc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import im2col_gemm_b200
    return im2col_gemm_b200


def normal(shape, dtype, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def near(got, want, bound):
    bound = bound + ref.half_step(want.abs() + bound, got.dtype)
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 7), (64, 64), (509, 777), (2, 3, 5, 7), (1000, 1024),
                                   (3, 1 << 20)])
def test_forward_and_backward(mqc, shape, dtype, residual):
    x, r = normal(shape, dtype), normal(shape, dtype, 1) if residual else None
    y = mqc.dropout_fwd(x, 0.3, SEED, OFFSET, residual=r)
    want, bound, keep = ref.dropout(x, 0.3, SEED, OFFSET, r)
    near(y, want, bound)
    if not residual:
        assert torch.equal(y != 0, keep & (x != 0))
    g = normal(shape, dtype, 2)
    want, bound, keep = ref.dropout(g, 0.3, SEED, OFFSET)
    gx = mqc.dropout_bwd(g, 0.3, SEED, OFFSET)
    near(gx, want, bound)
    assert torch.equal(gx != 0, keep & (g != 0))


@pytest.mark.parametrize("p", [0.0, 1e-6, 1.0 / 65536, 0.5, 0.99999, 1.0])
def test_probabilities(mqc, p):
    x = torch.ones(100, 1000, device="cuda")
    want, bound, keep = ref.dropout(x, p, SEED, 3)
    y = mqc.dropout_fwd(x, p, SEED, 3)
    near(y, want, bound)
    assert torch.equal(y != 0, keep)
    t = int(p * 65536 + 0.5)
    if t == 0:
        assert torch.equal(y, x)
    if t == 65536:
        assert not y.any()
    # the share dropped: a binomial of 100,000 draws, within six deviations
    q = t / 65536
    assert abs(1 - keep.double().mean().item() - q) <= 6 * (q * (1 - q) / 1e5) ** 0.5


def test_dropped_infinities_leave_nothing(mqc):
    x = torch.full((64, 64), float("inf"), device="cuda")
    x[0] = float("nan")
    y = mqc.dropout_fwd(x, 0.5, SEED)
    keep = ref.dropout(torch.ones_like(x), 0.5, SEED, 0)[2]
    assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols,gap", [(17, 40, 8), (17, 37, 3), (5, 8, 1), (300, 1000, 24), (6, 1, 4)])
def test_strides_and_untouched_gaps(mqc, rows, cols, gap, dtype):
    """The bits go by the logical index, not by the address; gaps stay."""
    x, r = normal((rows, cols), dtype), normal((rows, cols), dtype, 1)
    want = mqc.dropout_fwd(x, 0.4, SEED, OFFSET, residual=r)

    def wide(t):
        whole = torch.full((rows, cols + gap), 9.0, dtype=dtype, device="cuda")
        whole[:, :cols] = t
        return whole[:, :cols], whole
    out, whole = wide(torch.zeros_like(x))
    got = mqc.dropout_fwd(wide(x)[0], 0.4, SEED, OFFSET, residual=wide(r)[0], out=out)
    assert got is out and torch.equal(out, want) and (whole[:, cols:] == 9.0).all()
    assert torch.equal(mqc.dropout_fwd(wide(x)[0], 0.4, SEED, OFFSET, residual=r), want)   # some strided, some not
    assert torch.equal(mqc.dropout_bwd(wide(x)[0], 0.4, SEED, OFFSET), mqc.dropout_bwd(x, 0.4, SEED, OFFSET))


def test_in_place(mqc):
    x, r = normal((64, 100), BF16), normal((64, 100), BF16, 1)
    want = mqc.dropout_fwd(x, 0.25, SEED, residual=r)
    a, b = x.clone(), r.clone()
    assert torch.equal(mqc.dropout_fwd(a, 0.25, SEED, residual=r, out=a), want)
    assert torch.equal(mqc.dropout_fwd(x, 0.25, SEED, residual=b, out=b), want)


def test_seed_and_offset_choose_the_bits(mqc):
    x = torch.ones(256, 256, device="cuda")
    outs = [mqc.dropout_fwd(x, 0.5, s, o) for s, o in ((1, 0), (2, 0), (1, 1), (1 << 40, 0), (1, 1 << 40))]
    for i in range(len(outs)):
        for j in range(i):
            assert 0.4 < (outs[i] == outs[j]).double().mean() < 0.6


def test_a_captured_step_draws_new_bits(mqc):
    """offset_dev is read when the kernel runs: a replay after its advance uses
    the next bits, forward and backward alike."""
    x, g = normal((100, 130), BF16), normal((100, 130), BF16, 1)
    dev = torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mqc.dropout_fwd(x, 0.5, SEED, 10, offset_dev=dev)
        gx = mqc.dropout_bwd(g, 0.5, SEED, 10, offset_dev=dev)
        dev += 1
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, mqc.dropout_fwd(x, 0.5, SEED, 10 + step))
        assert torch.equal(gx, mqc.dropout_bwd(g, 0.5, SEED, 10 + step))


def test_empty(mqc):
    assert mqc.dropout_fwd(torch.empty(0, 5, device="cuda"), 0.5, 1).shape == (0, 5)
    assert mqc.dropout_bwd(torch.empty(5, 0, device="cuda"), 0.5, 1).shape == (5, 0)


def test_index_beyond_32_bits(mqc):
    """2^32 + 64 elements: the last ones take the blocks past 2^29, in a last
    row past a 32-bit offset."""
    cols = 64
    rows = (1 << 32) // cols + 1
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    x[-2:] = 1.0
    mqc.dropout_fwd(x, 0.5, SEED, OFFSET, out=x)
    n = 2 * cols
    bits = ref.dropout_bits(n, SEED, OFFSET, first=rows * cols - n)
    want = torch.from_numpy((bits >= 32768).astype("float32") * 2).view(2, cols)
    assert torch.equal(x[-2:].float().cpu(), want)


def test_helper_refusals(mqc):
    x = normal((8, 8), F32)
    for call in (lambda: mqc.dropout_fwd(x.t(), 0.5, 1), lambda: mqc.dropout_fwd(x, 0.5, 1, residual=x.to(BF16)),
                 lambda: mqc.dropout_fwd(x, 0.5, 1, residual=x[:4]), lambda: mqc.dropout_bwd(x, 0.5, 1, out=x[:4]),
                 lambda: mqc.dropout_fwd(x, 0.5, 1, offset_dev=x), lambda: mqc.dropout_fwd(x.cpu(), 0.5, 1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mqc.dropout_fwd(x.double(), 0.5, 1)


@pytest.mark.parametrize("which", ["x", "residual"])
def test_one_row_in_place_whatever_its_strides(mqc, which):
    """A single row has no next one: its strides may differ in place too."""
    n, seed = 1003, 77
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, r = (torch.randn(1, n, generator=gen, device="cuda") for _ in range(2))
    want = mqc.dropout_fwd(x, 0.25, seed, residual=r)
    y = x if which == "x" else r
    lds = (n + 5, n) if which == "x" else (n, n + 5)
    mqc.check(mqc.mqc_dropout_fwd(x.data_ptr(), lds[0], r.data_ptr(), lds[1], 1, n, mqc.F32, 0.25, seed, 0, None,
                                  y.data_ptr(), n, torch.cuda.current_stream().cuda_stream))
    assert torch.equal(y, want)
