"""Bounds of the dense layers' errors that hold where dense_ref's are wider
than the values themselves: far below zero, at large offsets, and in sums over
many pixels.

- The activations' errors are relative to their values.  SiLU is z q with q
  from a fast exponential and reciprocal: the exponent's rounding, |z| U, and a
  few steps more, and 0 where q is below the normal numbers.  GELU's normal
  distribution is P(t) exp(-z^2 / 2) below 0 and 1 minus that above: 2 U for the
  fit and its coefficients, 5 U for the evaluation of P, 6 U for t (a fused
  multiplication and a fast reciprocal, weighed by t P'/P <= 2), 4 U for the
  fast exponential, U for the product, and 1.5 z^2 U for the exponent's three
  roundings: (20 + 2 z^2) U of it; 0 where the exponential is below the normal
  numbers.
- Sums follow the longest chain of fp32 additions that the kernels have: `run`
  values that one thread adds up, and JOIN additions across the block (a
  thread's own channels, the rows of a block in turn, a warp's lanes); slabs
  and images are joined in fp64, the CTAs of a cluster (16 at most) in fp32.
- Each thread's mean is taken about its first value and has a rounding of the
  size of the values; the block's mean another JOIN of them.  The sums of
  squares are taken about these computed means, so that the means' errors
  enter the variance by twice their product with the deviation.
"""
import dense_ref as ref
import torch

NONE, RELU, SILU, GELU = 0, 1, 2, 3
U = ref.U
EPS = 1e-5
JOIN = 48
# Images that the two-pass form cuts into slabs, whose statistics and sums are
# joined: 256 groups of one channel side by side, one group, groups of two, few
# channels, several images.  A thread adds up 8 to 19 values of them, and no
# more than 100 where an image stays on chip (200 KB for at least 128 threads).
SLABS = [(1, 256, 180, 180, 256), (1, 64, 300, 300, 1), (2, 512, 60, 60, 256), (1, 8, 600, 600, 8),
         (4, 64, 160, 160, 16), (1, 16, 200, 200, 4)]
SLAB_PIXELS = [146, 203, 66, 1023, 231, 507]   # of one slab of each, fp32
RUN = 100


def make(n, c, h, w, dtype, seed=0, device="cpu", drift=False):
    """Channels-last inputs; drift: a mean of 1000 that moves by 8 down the
    image, so that the slabs have means of their own."""
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
    last = lambda t: t.to(dtype).permute(0, 3, 1, 2)  # noqa: E731
    x = r(n, h, w, c) + (torch.linspace(996.0, 1004.0, h, device=device).view(1, h, 1, 1) if drift else 0.5 * r(c))
    return dict(x=last(x), g=last(r(n, h, w, c)), gamma=1 + 0.2 * r(c), beta=0.3 * r(c))


def gelu_tail(z):
    """The normal distribution at -|z|, and what of it is flushed to 0."""
    tail = 0.5 * torch.special.erfc(z.abs() / 2 ** 0.5)
    return tail, torch.where(z.abs() > 13, tail, 0.0)


def act_error(z, a):
    """Error of act evaluated in fp32 at an exact z."""
    if a in (NONE, RELU):
        return torch.zeros_like(z)
    if a == GELU:
        tail, lost = gelu_tail(z)
        return z.abs() * (tail * ((20 + 2 * z * z) * U).clamp(max=1.0) + lost + U) * (z > 0) + (
            ref.act(z, a).abs() * ((21 + 2 * z * z) * U).clamp(max=1.0) + z.abs() * lost) * (z <= 0)
    y = ref.act(z, a).abs()
    return y * ((8 + 2 * z.abs()) * U).clamp(max=1.0) + torch.where(z < -86, y, 0.0)


def slope_error(z, a):
    """Error of act' evaluated in fp32 at an exact z."""
    if a in (NONE, RELU):
        return torch.zeros_like(z)
    if a == GELU:
        tail, lost = gelu_tail(z)
        bell = z.abs() * torch.exp(-z * z / 2) * (2 * torch.pi) ** -0.5
        return (tail + bell) * ((22 + 2 * z * z) * U).clamp(max=1.0) + lost * (1 + z.abs()) ** 2 + 2 * U * (z > 0)
    q = torch.sigmoid(z)
    return q * (1 + z.abs()) * ((8 + 2 * z.abs()) * U).clamp(max=1.0) + torch.where(z < -86, q * (1 + z.abs()), 0.0)


def act_spread(z, e, a):
    """How far act moves when z moves by e at most."""
    if a in (NONE, RELU):
        return e
    first = torch.maximum(ref.slope(z - e, a).abs(), ref.slope(z + e, a).abs()) * 1.02 + torch.where(
        z.abs() < 10, ref.CURVE[a] * e, 0.0)
    below = ref.act(z + e, a).abs()   # act rises to 0 towards -infinity
    return torch.where(e < 0.01, first * e, torch.where(z + e < -20, below, ref.LIP[a] * e))


def slope_spread(z, e, a):
    """How far act' moves when z moves by e at most (act'(z) = 1 - act'(-z))."""
    if a == NONE:
        return torch.zeros_like(z)
    if a == RELU:   # a sign that the error of z may flip
        return (z.abs() <= e).double()
    tail = ref.slope(-(z.abs() - e), a).abs()
    near = torch.where(z.abs() < 10, ref.CURVE[a] * e, (2 + z.abs() if a == GELU else 1.2) * tail * e)
    return torch.where(e < 0.01, near, torch.where(z.abs() - e > 20, tail, 2.2))


class GroupNorm(ref.GroupNorm):
    """Values and bounds of one group norm; run: values of a channel that one
    thread adds up (never more than the pixels)."""

    def __init__(self, x, groups, gamma, beta, eps, a, mean=None, rstd=None, run=None):
        super().__init__(x, groups, gamma, beta, eps, a, mean, rstd)
        n, c, h, w = x.shape
        self.run = h * w if run is None else run
        if mean is None:
            v = x.double().contiguous().view(n, groups, -1)
            var = (v - self.mean[..., None]).square().mean(2)
            wide, sigma = v.amax(2) - v.amin(2), (var + eps).sqrt()
            self.e_mean = U * (JOIN * v.abs().amax(2) + 2 * self.run * wide)
            off = self.e_mean / sigma
            self.e_rstd = self.rstd * (off + off.square() + (self.run + JOIN) * U * (wide / sigma).square() + 4 * U)
        dev = x.double() - self.spread(self.mean)
        self.e_xhat = self.spread(self.rstd) * (self.spread(self.e_mean) + U * dev.abs()) + (
            self.spread(self.e_rstd) * dev.abs()) + 2 * U * self.xhat.abs()
        self.e_z = self.gamma.abs() * self.e_xhat + 3 * U * ((self.xhat * self.gamma).abs() + self.beta.abs())

    def forward(self):
        return ref.act(self.z, self.a), act_spread(self.z, self.e_z, self.a) + act_error(self.z, self.a)

    def backward(self, g):
        """((gx, ggamma, gbeta), bounds)."""
        g, a = g.double(), self.a
        chain = self.run + JOIN
        es = slope_spread(self.z, self.e_z, a) + slope_error(self.z, a)
        dz = g * ref.slope(self.z, a)
        e = g.abs() * es + 2 * U * dz.abs()
        n, c, h, w = self.shape
        pixels, sp = (0, 2, 3), self.spread
        ggamma, gbeta = (dz * self.xhat).sum(pixels), dz.sum(pixels)
        prod = e * self.xhat.abs() + dz.abs() * self.e_xhat + 2 * U * (dz * self.xhat).abs()
        e_beta = e.sum(pixels) + chain * U * dz.abs().sum(pixels)
        e_gamma = prod.sum(pixels) + chain * U * (dz * self.xhat).abs().sum(pixels)
        grouped = lambda t: t.contiguous().view(n, self.groups, -1).sum(2) / self.count  # noqa: E731
        d, ed = dz * self.gamma, e * self.gamma.abs()
        k1, k2 = grouped(d), grouped(d * self.xhat)
        e1 = grouped(ed) + (chain + JOIN) * U * grouped(d.abs())
        e2 = grouped(prod * self.gamma.abs()) + (chain + JOIN) * U * grouped((d * self.xhat).abs())
        inner = d - sp(k1) - self.xhat * sp(k2)
        size = d.abs() + sp(k1).abs() + (self.xhat * sp(k2)).abs()
        e_in = ed + sp(e1) + self.xhat.abs() * sp(e2) + self.e_xhat * sp(k2).abs() + 6 * U * size
        e_gx = sp(self.rstd) * e_in + sp(self.e_rstd) * inner.abs() + U * (sp(self.rstd) * inner).abs()
        return (sp(self.rstd) * inner, ggamma, gbeta), (e_gx, e_gamma, e_beta)


def outside(got, want, bound, dtype):
    """Where a result is further from its value than the bound and the final rounding allow (NaN: where it is no NaN)."""
    allowed = bound + ref.half_step(want.abs() + bound, dtype)
    return torch.where(torch.isnan(want), ~torch.isnan(got), ~((got.double() - want).abs() <= allowed))
