"""The dense layers together, as a network uses them: a convolution of the
library, then the residual branch  y = x + dropout(act-linear(act(group_norm(
x))))  over its pixels, forward and backward, against float64."""
import dense_ref as ref
import pytest
import torch

pytestmark = pytest.mark.gpu
SEED, P = 1234567, 0.2


@pytest.fixture(scope="module")
def mqc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import im2col_gemm_b200
    return im2col_gemm_b200


class Branch:
    """out = x + dropout(silu(x' W1^T + b1) W2^T + b2), x' = silu(group_norm(x)),
    over a channels-last x [N][C][H][W]; the backward pass draws the mask again."""

    def __init__(self, mqc, c, hidden, groups, dtype, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.mqc, self.groups = mqc, groups
        self.gamma, self.beta = 1 + 0.1 * r(c), 0.1 * r(c)
        self.w1, self.b1 = (r(hidden, c) * c ** -0.5).to(dtype), 0.1 * r(hidden)
        self.w2, self.b2 = (r(c, hidden) * hidden ** -0.5).to(dtype), 0.1 * r(c)

    def tokens(self, t):
        n, c, h, w = t.shape
        return t.permute(0, 2, 3, 1).reshape(n * h * w, c)

    def image(self, t, like):
        n, c, h, w = like.shape
        return t.view(n, h, w, c).permute(0, 3, 1, 2)

    def forward(self, x, offset):
        m = self.mqc
        self.x, self.offset = x, offset
        self.h, self.mean, self.rstd = m.group_norm_fwd(x, self.groups, self.gamma, self.beta, 1e-5, m.ACT_SILU)
        self.u, self.z = m.linear_fwd(self.tokens(self.h), self.w1, self.b1, m.ACT_SILU, save_z=True)
        v, _ = m.linear_fwd(self.u, self.w2, self.b2)
        return self.image(m.dropout_fwd(v, P, SEED, offset, residual=self.tokens(x)), x)

    def backward(self, g):
        m = self.mqc
        gv = m.dropout_bwd(self.tokens(g), P, SEED, self.offset)
        gu, gw2, gb2 = m.linear_bwd(gv, self.u, self.w2)
        gh, gw1, gb1 = m.linear_bwd(gu, self.tokens(self.h), self.w1, self.z, m.ACT_SILU)
        gx, ggamma, gbeta = m.group_norm_bwd(self.image(gh, g), self.x, self.groups, self.mean, self.rstd, self.gamma,
                                             self.beta, m.ACT_SILU)
        return gx + g, ggamma, gbeta, gw1, gb1, gw2, gb2

    def exact(self, x, g, offset):
        """Output and gradients in float64 by autograd."""
        leaf = lambda t: t.double().detach().requires_grad_(True)  # noqa: E731
        xs = leaf(x.contiguous())
        ps = [leaf(t) for t in (self.gamma, self.beta, self.w1, self.b1, self.w2, self.b2)]
        gamma, beta, w1, b1, w2, b2 = ps
        h = torch.nn.functional.silu(torch.group_norm(xs, self.groups, gamma, beta, 1e-5))
        u = torch.nn.functional.silu(self.tokens(h) @ w1.t() + b1)
        v = u @ w2.t() + b2
        keep = ref.dropout(torch.ones(v.shape, device=v.device), P, SEED, offset)[0]
        out = xs + self.image(v * keep, xs)
        out.backward(g.double())
        return out.detach(), [t.grad for t in [xs] + ps]


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


# every tensor of the chain is rounded once: at most seven roundings of half a
# step (2^-8 for bf16, 2^-11 for fp16) reach an output, each at worst at its
# full size
LIMIT = {torch.bfloat16: 7 * 2.0 ** -8, torch.float16: 7 * 2.0 ** -11}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(2, 64, 20, 20, 8, 128), (3, 40, 7, 9, 5, 100), (16, 128, 40, 40, 32, 256)])
def test_residual_branch(mqc, shape, dtype):
    n, c, h, w, groups, hidden = shape
    b = Branch(mqc, c, hidden, groups, dtype)
    gen = torch.Generator(device="cuda").manual_seed(5)
    img = lambda: torch.randn(n, h, w, c, generator=gen, device="cuda").to(dtype).permute(0, 3, 1, 2)  # noqa: E731
    x, g = img(), img()
    out = b.forward(x, 3)
    grads = b.backward(g)
    mqc.check(mqc.get_device_status())
    want, wgrads = b.exact(x, g, 3)
    assert rel(out, want) <= LIMIT[dtype]
    for a, e in zip(grads, wgrads):
        assert rel(a, e) <= LIMIT[dtype]


def test_branch_after_a_quantized_convolution(mqc, orc):
    """conv2d_fwd (MXFP8) -> branch -> the next layer's quantizer: the branch
    takes the convolution's own fp32 output and its result quantizes to the
    codes that the oracle gives for the same values."""
    n, c, hw, k = 16, 32, 16, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(n, c, hw, hw, generator=gen, device="cuda")
    w = torch.randn(k, c, 3, 3, generator=gen, device="cuda") * 0.05
    cv = mqc.conv_desc(n, c, hw, hw, k, 3, 3, 1, 1)
    q = lambda t: mqc.quantize_mx(t, mqc.E4M3, mqc.SQ32, mqc.ORDER_BA)  # noqa: E731
    y = mqc.conv2d_fwd(q(x), q(w), cv)
    y = y.to(memory_format=torch.channels_last)
    h, mean, rstd = mqc.group_norm_fwd(y, 8, act=mqc.ACT_SILU)
    r = ref.GroupNorm(y, 8, None, None, 1e-5, mqc.ACT_SILU)
    want, bound = r.forward()
    assert ((h.double() - want).abs() <= bound + ref.half_step(want.abs() + bound, torch.float32)).all()
    out = Branch(mqc, k, 128, 8, torch.bfloat16).forward(h.to(torch.bfloat16), 0).float()
    codes = mqc.quantize_mx(out, mqc.E4M3, mqc.SQ32, mqc.ORDER_BA)
    mqc.check(mqc.get_device_status())
    rc, rs = orc.quantize(out.contiguous().cpu().numpy(), 0, 2, 0)
    assert (codes.codes.cpu().numpy() == rc).all() and (codes.scales.cpu().numpy() == rs).all()


def test_a_captured_training_step(mqc):
    """Forward and backward of the branch in one graph: the replay equals the
    eager calls bit for bit, on new inputs too."""
    b = Branch(mqc, 64, 128, 8, torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(6)
    img = lambda: torch.randn(4, 20, 20, 64, generator=gen, device="cuda").to(torch.bfloat16).permute(0, 3, 1, 2)  # noqa: E731
    x, g = img(), img()
    step = lambda: [b.forward(x, 9)] + list(b.backward(g))  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        x.copy_(img())
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(got, step()):
            assert torch.equal(a, e)
