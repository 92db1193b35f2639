"""Plain 64-bit forms of the dense layers (group norm with an activation,
linear, dropout) and the rounding bounds their tests use.

The forms are the formulas of include/mqc.h in float64 (torch; numpy integers
for the generator).  The bounds follow the kernels' arithmetic:
- a rounding to type T is off by at most half a step, eps(T)/2 relative, or
  half a subnormal step;
- an fp32 operation is off by at most U = 2^-24 relative, and the fast
  exponential and division of SiLU by (8 + 2|z|) steps of it;
- a sum of n terms in fp32, in any order, by at most n U sum|term|; in the
  tensor cores 16 products enter an accumulation step, whose rounding may be a
  truncation (2 U), so a product over K by (K/16 + 16 + 8) 2 U sum|ab|.
"""
import math

import numpy as np
import torch

NONE, RELU, SILU, GELU = 0, 1, 2, 3
U = 2.0 ** -24
LIP = {NONE: 1.0, RELU: 1.0, SILU: 1.1, GELU: 1.13}       # max |act'|
CURVE = {NONE: 0.0, RELU: 0.0, SILU: 0.5, GELU: 0.8}      # max |act''|


def half_step(v, dtype):
    """Half a step of `dtype` at the values v (float64)."""
    tiny = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}[dtype]
    return v.abs() * (torch.finfo(dtype).eps / 2) + tiny


def act(z, a):
    if a == RELU:
        return torch.where(z < 0, torch.zeros_like(z), z)
    if a == SILU:
        return z * torch.sigmoid(z)
    if a == GELU:
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    return z


def slope(z, a):
    if a == RELU:
        return (z > 0).double()
    if a == SILU:
        q = torch.sigmoid(z)
        return q + z * q * torch.sigmoid(-z)
    if a == GELU:
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def act_error(z, a):
    """Error of act evaluated in fp32 at an exact z."""
    return 0.0 if a in (NONE, RELU) else (8 + 2 * z.abs()) * U * z.abs()


def slope_error(z, a):
    """Error of act' evaluated in fp32 at an exact z: a few operations on values up to 1 + |z|."""
    return 0.0 if a in (NONE, RELU) else (8 + 2 * z.abs()) * U * (1 + z.abs())


# ------------------------------------------------------------------ linear
def product_error(a, b):
    """Bound of a . b^T in the tensor cores (a [I][R], b [J][R], float64)."""
    return (a.shape[1] / 16 + 24) * 2 * U * (a.abs() @ b.abs().t())


def linear_fwd(x, w, bias, a, residual):
    """(y, z, bound of y, bound of z) before the final roundings."""
    x, w = x.double(), w.double()
    z, ez = x @ w.t(), product_error(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * (z.abs() + bias.double().abs())
    y, ey = act(z, a), LIP[a] * ez + act_error(z, a)
    if residual is not None:
        y = y + residual.double()
        ey = ey + U * y.abs()
    return y, z, ey, ez


def linear_bwd(g, x, w, z, a):
    """((gx, gw, gb), their bounds before the final rounding): dz enters the
    products rounded to the operand type."""
    t = g.dtype
    g, x, w = g.double(), x.double(), w.double()
    dz, e = g, torch.zeros_like(g)
    if a != NONE:
        dz = g * slope(z.double(), a)
        e = g.abs() * slope_error(z.double(), a) + 2 * U * dz.abs()
    er = e + (half_step(dz, t) if a not in (NONE, RELU) else 0.0)
    gx, gw, gb = dz @ w, dz.t() @ x, dz.sum(0)
    ex = er @ w.abs() + product_error(dz, w.t())
    ew = er.t() @ x.abs() + product_error(dz.t(), x.t())
    eb = e.sum(0) + g.shape[0] * U * dz.abs().sum(0)
    return (gx, gw, gb), (ex, ew, eb)


# ------------------------------------------------------------------ group norm
class GroupNorm:
    """Values and bounds of one group norm, x [N][C][H][W]."""

    def __init__(self, x, groups, gamma, beta, eps, a, mean=None, rstd=None):
        n, c, h, w = x.shape
        self.shape, self.groups, self.a = x.shape, groups, a
        v = x.double().contiguous().view(n, groups, -1)
        count, seq = v.shape[2], h * w + 16
        self.mean = v.mean(2)
        var = (v - self.mean[..., None]).square().mean(2)
        self.rstd = (var + eps).rsqrt()
        # fp32 mean and deviations: at most one rounding a step of size U max|x|
        top = v.abs().amax(2)
        self.e_mean = seq * U * top
        e_var = 2 * self.e_mean * var.sqrt() + self.e_mean.square() + seq * 2 * U * var
        self.e_rstd = self.rstd * (0.5 * e_var / (var + eps) + 2 * U)
        if mean is not None:   # the statistics are given: exact inputs
            self.mean, self.rstd = mean.double(), rstd.double()
            self.e_mean, self.e_rstd = torch.zeros_like(self.mean), torch.zeros_like(self.rstd)
        spread = lambda s: s.repeat_interleave(c // groups, 1).view(n, c, 1, 1)  # noqa: E731
        self.spread, self.count = spread, count
        per = lambda p, d: (p.double() if p is not None else torch.full((c,), d, dtype=torch.float64,  # noqa: E731
                                                                       device=x.device)).view(1, c, 1, 1)
        self.gamma, self.beta = per(gamma, 1.0), per(beta, 0.0)
        dev = x.double() - spread(self.mean)
        self.xhat = dev * spread(self.rstd)
        self.e_xhat = spread(self.rstd) * (spread(self.e_mean) + U * dev.abs()) + (
            spread(self.e_rstd) * dev.abs()) + 2 * U * self.xhat.abs()
        self.z = self.xhat * self.gamma + self.beta
        self.e_z = self.gamma.abs() * self.e_xhat + 3 * U * ((self.xhat * self.gamma).abs() + self.beta.abs())

    def forward(self):
        return act(self.z, self.a), LIP[self.a] * self.e_z + act_error(self.z, self.a)

    def backward(self, g):
        """((gx, ggamma, gbeta), bounds)."""
        g = g.double()
        s = slope(self.z, self.a)
        if self.a == RELU:   # a sign that the error of z may flip
            es = (self.z.abs() <= self.e_z).double()
        else:
            es = CURVE[self.a] * self.e_z + slope_error(self.z, self.a)
        dz = g * s
        e = g.abs() * es + 2 * U * dz.abs()
        n, c, h, w = self.shape
        n_sum = n * h * w
        gb, ggam = dz.sum((0, 2, 3)), (dz * self.xhat).sum((0, 2, 3))
        eb = e.sum((0, 2, 3)) + n_sum * U * dz.abs().sum((0, 2, 3))
        prod = e * self.xhat.abs() + dz.abs() * self.e_xhat + 2 * U * (dz * self.xhat).abs()
        eg = prod.sum((0, 2, 3)) + n_sum * U * (dz * self.xhat).abs().sum((0, 2, 3))
        grouped = lambda t: t.contiguous().view(n, self.groups, -1).sum(2) / self.count  # noqa: E731
        d, ed = dz * self.gamma, e * self.gamma.abs()
        k1, k2 = grouped(d), grouped(d * self.xhat)
        seq = h * w + 16
        e1 = grouped(ed) + seq * U * grouped(d.abs())
        e2 = grouped(prod * self.gamma.abs()) + seq * U * grouped((d * self.xhat).abs())
        sp = self.spread
        inner = d - sp(k1) - self.xhat * sp(k2)
        size = d.abs() + sp(k1).abs() + (self.xhat * sp(k2)).abs()
        e_in = ed + sp(e1) + self.xhat.abs() * sp(e2) + self.e_xhat * sp(k2).abs() + 6 * U * size
        gx = sp(self.rstd) * inner
        return (gx, ggam, gb), (sp(self.rstd) * e_in + sp(self.e_rstd) * inner.abs() + U * gx.abs(), eg, eb)


# ------------------------------------------------------------------ dropout
def philox4x32_10(counter, key):
    """Blocks of Philox4x32-10: counter [n][4], key (k0, k1) -> [n][4] uint32."""
    c = [np.asarray(counter[:, i], dtype=np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    lo, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> half) ^ c[1] ^ np.uint64(k0), q & lo, (p >> half) ^ c[3] ^ np.uint64(k1), p & lo]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).astype(np.uint32)


def dropout_bits(n, seed, offset, first=0):
    """The 16 random bits of elements first .. first + n - 1 (first a multiple of 8)."""
    b = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    lo = np.uint64(0xFFFFFFFF)
    counter = np.stack([b & lo, b >> np.uint64(32), np.full_like(b, offset & 0xFFFFFFFF),
                        np.full_like(b, (offset >> 32) & 0xFFFFFFFF)], 1)
    w = philox4x32_10(counter, (seed & 0xFFFFFFFF, seed >> 32))
    return np.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]


def dropout(x, p, seed, offset, residual=None):
    """(y, bound before the final rounding) for a matrix or contiguous x."""
    t = int(math.floor(p * 65536 + 0.5))
    keep = torch.from_numpy(dropout_bits(x.numel(), seed, offset).astype(np.int64) >= t).view(x.shape).to(x.device)
    scale = 65536 / (65536 - t) if t < 65536 else 0.0
    y = torch.where(keep, x.double() * scale, torch.zeros_like(x, dtype=torch.float64))
    e = 2 * U * y.abs()
    if residual is not None:
        y = y + residual.double()
        e = e + U * y.abs()
    return y, e, keep
