"""Cases of the dense-layer operators (group norm with an activation, linear
with bias, activation and residual, dropout from a counter-based generator),
with their plain forms in elementary torch operations and their values in 64
bits."""
import math

import numpy as np
import torch

own = False

# The activations' codes of the library (mqc_act).
NONE, RELU, SILU, GELU = 0, 1, 2, 3
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


# ------------------------------------------------------------------ cases
def _gn(name, op, n, c, h, w, groups, dtype, act):
    return {"name": name, "op": op, "n": n, "c": c, "h": h, "w": w, "groups": groups, "dtype": dtype, "act": act}


def _lin(name, op, m, n, k, dtype, act, bias=True, residual=False, save_z=False):
    return {"name": name, "op": op, "m": m, "n": n, "k": k, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "save_z": save_z}


def _drop(name, op, rows, cols, dtype, p, residual=False):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "p": p, "residual": residual}


def listed():
    return [
        # one image of the latent-replay block's input in inference: latency
        _gn("gn fwd 1 image", "gn_fwd", 1, 256, 14, 14, 32, "bf16", SILU),
        # layer 2 of the YOLOv8n-shaped stack in training: more than the L2 cache holds
        _gn("gn fwd yolo 160", "gn_fwd", 16, 64, 160, 160, 16, "bf16", SILU),
        # odd spatial size, groups of 10 channels, full precision
        _gn("gn fwd odd f32", "gn_fwd", 7, 320, 45, 37, 32, "f32", RELU),
        # the latent-replay block in training
        _gn("gn bwd latent", "gn_bwd", 128, 256, 14, 14, 32, "bf16", SILU),
        # a large-batch layer in training, full precision
        _gn("gn bwd large f32", "gn_bwd", 32, 128, 80, 80, 32, "f32", SILU),
        # a head on one token: the weights are read once
        _lin("linear fwd 1 token", "linear_fwd", 1, 4096, 4096, "bf16", SILU, residual=True),
        # a classifier over the features of one batch, odd number of classes
        _lin("linear fwd classes", "linear_fwd", 128, 1003, 515, "f16", NONE),
        # a wide layer over the tokens of a batch, in training
        _lin("linear fwd wide", "linear_fwd", 8192, 4096, 4096, "bf16", GELU, residual=True, save_z=True),
        # its narrower gradient
        _lin("linear bwd wide", "linear_bwd", 8192, 2048, 2048, "bf16", SILU),
        # the gradient of an odd layer over few tokens
        _lin("linear bwd odd", "linear_bwd", 509, 777, 1003, "f16", RELU),
        # the branch's output dropped and added to the skip path
        _drop("dropout fwd add", "dropout_fwd", 16384, 2048, "bf16", 0.1, residual=True),
        # the gradient of a small odd layer
        _drop("dropout bwd odd", "dropout_bwd", 509, 777, "f32", 0.3),
    ]


MOST = {"bytes": 700e6, "flops": 270e9}  # a drawn case stays within the largest listed ones


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["gn_fwd", "gn_bwd", "linear_fwd", "linear_bwd", "dropout_fwd", "dropout_bwd"])
    if op.startswith("gn"):
        groups = rng.choice([1, 2, 4, 8, 16, 32])
        per = max(1, _log(rng, max(1, 16 // groups), 1024 // groups))
        return _gn("", op, _log(rng, 1, 64), groups * per, _log(rng, 1, 200), _log(rng, 1, 200), groups,
                   rng.choice(["f32", "bf16", "f16"]), rng.choice([NONE, RELU, SILU, GELU]))
    if op.startswith("linear"):
        size = lambda: _log(rng, 16, 6000) if rng.random() < 0.5 else 8 * _log(rng, 2, 750)  # noqa: E731
        return _lin("", op, _log(rng, 1, 12000), size(), size(), rng.choice(["bf16", "f16"]),
                    rng.choice([NONE, RELU, SILU, GELU]), rng.random() < 0.7,
                    op == "linear_fwd" and rng.random() < 0.5, op == "linear_fwd" and rng.random() < 0.3)
    return _drop("", op, _log(rng, 1, 20000), _log(rng, 1, 5000), rng.choice(["f32", "bf16", "f16"]),
                 rng.choice([0.05, 0.1, 0.25, 0.5]), op == "dropout_fwd" and rng.random() < 0.5)


def draw(rng):
    while True:
        case = _drawn(rng)
        w = work(case)
        if 1e5 < w["bytes"] < MOST["bytes"] and w["flops"] < MOST["flops"]:
            del case["name"]
            return case


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "f32" else 2
    if op.startswith("gn"):
        n = case["n"] * case["c"] * case["h"] * case["w"]
        return {"bytes": n * size * (2 if op == "gn_fwd" else 3) + 8 * case["c"] + 8 * case["n"] * case["groups"],
                "flops": n * (12 if op == "gn_fwd" else 24)}
    if op.startswith("linear"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "linear_fwd":
            moved = m * k + n * k + m * n * (1 + case["residual"] + case["save_z"])
            return {"bytes": moved * size + 4 * n * case["bias"], "flops": 2 * m * n * k}
        moved = 2 * m * k + 2 * n * k + m * n * (1 + (case["act"] != NONE))
        return {"bytes": moved * size + 4 * n * case["bias"], "flops": 4 * m * n * k}
    n = case["rows"] * case["cols"]
    return {"bytes": n * size * (2 + case["residual"]), "flops": n * 12}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, to=t):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(to)

    op, s = case["op"], {"case": dict(case)}
    if op.startswith("gn"):
        n, c, h, w, groups = (case[k] for k in ("n", "c", "h", "w", "groups"))
        # a convolution's outputs: every channel with its own offset and spread
        x = torch.randn(n, h, w, c, generator=gen, device="cuda")
        x = x * (0.5 + torch.rand(c, generator=gen, device="cuda")) + torch.randn(c, generator=gen, device="cuda")
        s["x"] = x.to(t).permute(0, 3, 1, 2)
        s["gamma"] = 1 + normal(c, scale=0.1, to=torch.float32)
        s["beta"] = normal(c, scale=0.1, to=torch.float32)
        if op == "gn_bwd":
            # the incoming gradient, and what the forward pass kept
            s["g"] = normal(n, h, w, c, scale=0.1).permute(0, 3, 1, 2)
            v = s["x"].reshape(n, groups, -1).double()
            s["mean"] = v.mean(2).float()
            s["rstd"] = (v.var(2, unbiased=False) + EPS).rsqrt().float()
    elif op.startswith("linear"):
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = normal(m, k)
        s["w"] = normal(n, k, scale=k ** -0.5)
        if op == "linear_fwd":
            s["bias"] = normal(n, scale=0.1, to=torch.float32) if case["bias"] else None
            s["residual"] = normal(m, n) if case["residual"] else None
        else:
            s["g"] = normal(m, n, scale=0.1)
            s["z"] = normal(m, n) if case["act"] != NONE else None
    else:
        s["x"] = normal(case["rows"], case["cols"])
        s["residual"] = normal(case["rows"], case["cols"]) if case["residual"] else None
        s["seed"], s["offset"] = (seed * 0x9E3779B97F4A7C15 + 1) % 2 ** 64, seed % 1000
    return s


# ------------------------------------------------------------------ plain forms
def _act(z, act):
    if act == RELU:
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == SILU:
        return z / (1 + torch.exp(-z))
    if act == GELU:
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _dact(z, act):
    if act == RELU:
        return (z > 0).to(z.dtype)
    if act == SILU:
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if act == GELU:
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return torch.ones_like(z)


def _rows(x, groups):
    """[N][C][H][W] in memory order [N][H W][G][D], in 32 bits."""
    n, c, h, w = x.shape
    return x.permute(0, 2, 3, 1).reshape(n, h * w, groups, c // groups).float()


def _image(v, like):
    n, c, h, w = like.shape
    return v.reshape(n, h, w, c).to(like.dtype).permute(0, 3, 1, 2)


def _gn_fwd(s, case):
    x, groups = s["x"], case["groups"]
    v = _rows(x, groups)
    mean = v.mean((1, 3), keepdim=True)
    d = v - mean
    rstd = torch.rsqrt((d * d).mean((1, 3), keepdim=True) + EPS)
    z = d * rstd * s["gamma"].view(groups, -1) + s["beta"].view(groups, -1)
    return _image(_act(z, case["act"]), x), mean.reshape(-1, groups), rstd.reshape(-1, groups)


def _gn_bwd(s, case):
    x, groups = s["x"], case["groups"]
    gamma, beta = s["gamma"].view(groups, -1), s["beta"].view(groups, -1)
    rstd = s["rstd"].view(-1, 1, groups, 1)
    xhat = (_rows(x, groups) - s["mean"].view(-1, 1, groups, 1)) * rstd
    dz = _rows(s["g"], groups) * _dact(xhat * gamma + beta, case["act"])
    dgamma, dbeta = (dz * xhat).sum((0, 1)), dz.sum((0, 1))
    d = dz * gamma
    dx = rstd * (d - d.mean((1, 3), keepdim=True) - xhat * (d * xhat).mean((1, 3), keepdim=True))
    return _image(dx, x), dgamma.reshape(-1), dbeta.reshape(-1)


def _linear_fwd(s, case):
    z = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    t = s["x"].dtype
    return [y.to(t), z.to(t)] if case["save_z"] else [y.to(t)]


def _linear_bwd(s, case):
    t, dz = s["x"].dtype, s["g"].float()
    if s["z"] is not None:
        dz = dz * _dact(s["z"].float(), case["act"])
    out = [torch.matmul(dz, s["w"].float()).to(t), torch.matmul(dz.t(), s["x"].float()).to(t)]
    return out + [dz.sum(0)] if case["bias"] else out


def _random16(n, seed, offset):
    """16 random bits for each of n elements: Philox4x32-10 with key `seed` and
    counter (element / 8, offset), eight halves a block."""
    low = 0xFFFFFFFF
    block = torch.arange((n + 7) // 8, device="cuda")
    c = [block & low, block >> 32, torch.full_like(block, offset & low), torch.full_like(block, offset >> 32)]
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # the low 64 bits, which hold both halves
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, 1)
    return torch.stack((words & 0xFFFF, words >> 16), 2).reshape(-1)[:n]


def _dropout(s, case):
    x = s["x"]
    t = round(case["p"] * 65536)
    keep = (_random16(x.numel(), s["seed"], s["offset"]) >= t).view(x.shape)
    y = torch.where(keep, x.float() * (65536 / (65536 - t)), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(x.dtype)


def _own(s, case):
    import im2col_gemm_b200 as mqc
    op = case["op"]
    if op == "gn_fwd":
        return mqc.group_norm_fwd(s["x"], case["groups"], s["gamma"], s["beta"], EPS, case["act"])
    if op == "gn_bwd":
        return mqc.group_norm_bwd(s["g"], s["x"], case["groups"], s["mean"], s["rstd"], s["gamma"], s["beta"],
                                  case["act"])
    if op == "linear_fwd":
        y, z = mqc.linear_fwd(s["x"], s["w"], s["bias"], case["act"], s["residual"], save_z=case["save_z"])
        return [y, z] if case["save_z"] else [y]
    if op == "linear_bwd":
        gx, gw, gb = mqc.linear_bwd(s["g"], s["x"], s["w"], s["z"], case["act"], need_bias=case["bias"])
        return [gx, gw, gb] if case["bias"] else [gx, gw]
    if op == "dropout_fwd":
        return mqc.dropout_fwd(s["x"], case["p"], s["seed"], s["offset"], residual=s["residual"])
    return mqc.dropout_bwd(s["x"], case["p"], s["seed"], s["offset"])


PLAIN = {"gn_fwd": _gn_fwd, "gn_bwd": _gn_bwd, "linear_fwd": _linear_fwd, "linear_bwd": _linear_bwd,
         "dropout_fwd": _dropout, "dropout_bwd": _dropout}


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return PLAIN[case["op"]](state, case)


# ------------------------------------------------------------------ values in 64 bits
def _sigma(z, act):
    """(act(z), act'(z)) in 64 bits."""
    if act == RELU:
        return z.clamp(min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if act == SILU:
        q = torch.sigmoid(z)
        return z * q, q + z * q * torch.sigmoid(-z)
    if act == GELU:
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def _exact_gn(s, case):
    n, c, h, w = s["x"].shape
    groups = case["groups"]
    per_channel = lambda v: v.double().view(1, c, 1)  # noqa: E731
    spread = lambda v: v.double().repeat_interleave(c // groups, 1).view(n, c, 1)  # noqa: E731
    grouped = lambda v: v.view(n, groups, -1).mean(2)  # noqa: E731
    x = s["x"].double().contiguous().view(n, c, h * w)
    if case["op"] == "gn_fwd":
        mean = grouped(x)
        var = grouped((x - spread(mean)).square())
        rstd = 1 / torch.sqrt(var + EPS)
        z = torch.addcmul(per_channel(s["beta"]), (x - spread(mean)) * spread(rstd), per_channel(s["gamma"]))
        return _sigma(z, case["act"])[0].view(n, c, h, w), mean, rstd
    xhat = (x - spread(s["mean"])) * spread(s["rstd"])
    slope = _sigma(xhat * per_channel(s["gamma"]) + per_channel(s["beta"]), case["act"])[1]
    dz = s["g"].double().contiguous().view(n, c, h * w) * slope
    down = dz * per_channel(s["gamma"])
    a, b = grouped(down), grouped(down * xhat)
    dx = (down - spread(a) - xhat * spread(b)) * spread(s["rstd"])
    return dx.view(n, c, h, w), torch.einsum("ncp,ncp->c", dz, xhat), torch.einsum("ncp->c", dz)


def _exact_linear(s, case):
    x, w = s["x"].double(), s["w"].double()
    if case["op"] == "linear_fwd":
        z = torch.einsum("mk,nk->mn", x, w)
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _sigma(z, case["act"])[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return [y, z] if case["save_z"] else [y]
    dz = s["g"].double()
    if s["z"] is not None:
        dz = dz * _sigma(s["z"].double(), case["act"])[1]
    out = [torch.einsum("mn,nk->mk", dz, w), torch.einsum("mn,mk->nk", dz, x)]
    return out + [torch.einsum("mn->n", dz)] if case["bias"] else out


def _exact_dropout(s, case):
    """The generator once more, with numpy's unsigned integers on the host."""
    n = s["x"].numel()
    at = np.arange(-(-n // 8), dtype=np.uint64)
    mask, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    x0, x1 = at & mask, at >> half
    x2 = np.full_like(at, s["offset"] & 0xFFFFFFFF)
    x3 = np.full_like(at, s["offset"] >> 32)
    keys = [((s["seed"] + i * 0x9E3779B9) & 0xFFFFFFFF, ((s["seed"] >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)
            for i in range(10)]
    for lo, hi in keys:
        p, q = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = (q >> half) ^ x1 ^ np.uint64(lo), q & mask, (p >> half) ^ x3 ^ np.uint64(hi), p & mask
    bits = np.stack([x0, x1, x2, x3], 1).astype("<u4").view("<u2").reshape(-1)[:n]
    drop = int(math.floor(case["p"] * 65536 + 0.5))
    keep = torch.from_numpy(bits.astype(np.int32) >= drop).to("cuda").view(s["x"].shape)
    y = keep * s["x"].double() * 65536 / (65536 - drop)
    return y if s["residual"] is None else y + s["residual"].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("gn"):
        return _exact_gn(s, case)
    if case["op"].startswith("linear"):
        return _exact_linear(s, case)
    return _exact_dropout(s, case)
