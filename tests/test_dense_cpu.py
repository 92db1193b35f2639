"""CPU tests of the dense layers: the argument checks of their entry points
(nothing is launched), workspace sizes, and the 64-bit forms that the GPU
tests compare with (known answers of the generator; gradients against central
differences of the forward forms)."""
import ctypes

import dense_ref as ref
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def mqc():
    import __graft_entry__
    __graft_entry__.build()
    import im2col_gemm_b200
    return im2col_gemm_b200


P16 = ctypes.c_void_p(256)      # never read: every call below is refused or writes nothing
ODD = ctypes.c_void_p(260)


def test_philox_known_answers():
    """Vectors published with the generator (Salmon et al., Random123)."""
    cases = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
             ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
             ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
              (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for counter, key, want in cases:
        got = ref.philox4x32_10(np.array([counter], dtype=np.uint64), key)
        assert tuple(int(v) for v in got[0]) == want


def test_dropout_bits_place():
    """Element i takes half i % 2 of word (i % 8) / 2 of block i / 8."""
    w = ref.philox4x32_10(np.array([[3, 0, 5, 2]], dtype=np.uint64), (7, 9))[0]
    bits = ref.dropout_bits(32, 7 | (9 << 32), 5 | (2 << 32))
    for e in range(8):
        assert int(bits[24 + e]) == (int(w[e // 2]) >> (16 * (e % 2))) & 0xFFFF


@pytest.mark.parametrize("a", [0, 1, 2, 3])
def test_activation_slopes_against_differences(a):
    z = torch.linspace(-6, 6, 1001, dtype=torch.float64) + 1e-3   # away from ReLU's corner
    h = 1e-6
    diff = (ref.act(z + h, a) - ref.act(z - h, a)) / (2 * h)
    # third derivative below 2: h^2/6 * 2, and cancellation 2^-52 |act| / h
    assert (diff - ref.slope(z, a)).abs().max() < 1e-8


@pytest.mark.parametrize("a", [0, 1, 2, 3])
def test_linear_gradient_against_differences(a):
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, b, g = r(5, 7), r(4, 7), r(4), r(5, 4)
    z = ref.linear_fwd(x, w, b, a, None)[1]
    # float64 has no entry among the rounded types: the values alone are wanted
    dz = g * ref.slope(z, a)
    grads = {"x": dz @ w, "w": dz.t() @ x, "b": dz.sum(0)}
    h = 1e-6
    for name, v in (("x", x), ("w", w), ("b", b)):
        d = r(*v.shape)
        at = lambda s: ref.linear_fwd(*(t + s * h * d if n == name else t  # noqa: E731
                                        for n, t in (("x", x), ("w", w), ("b", b))), a, None)[0]
        diff = ((at(1) - at(-1)) * g).sum() / (2 * h)
        assert abs(diff - (grads[name] * d).sum()) < 1e-6 * (1 + abs(diff))


@pytest.mark.parametrize("a", [0, 1, 2, 3])
def test_group_norm_gradient_against_differences(a):
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, gamma, beta, g = r(2, 6, 3, 4), r(6), r(6), r(2, 6, 3, 4)
    grads = ref.GroupNorm(x, 3, gamma, beta, 1e-3, a).backward(g)[0]
    h = 1e-6
    for i, v in enumerate((x, gamma, beta)):
        d = r(*v.shape)
        at = lambda s: ref.GroupNorm(*[(t + s * h * d if j == i else t) if j != 1 else 3  # noqa: E731
                                       for j, t in ((0, x), (1, None))],
                                     gamma + s * h * d if i == 1 else gamma,
                                     beta + s * h * d if i == 2 else beta, 1e-3, a).forward()[0]
        diff = ((at(1) - at(-1)) * g).sum() / (2 * h)
        assert abs(diff - (grads[i] * d).sum()) < 1e-6 * (1 + abs(diff))


def test_linear_refusals(mqc):
    lin = lambda **k: mqc.Linear(**{**dict(M=4, N=8, K=16, dtype=1, act=0, ldx=16, ldw=16, ldr=8, ldy=8, ldz=8,  # noqa: E731
                                          ldg=8, ldgx=16, ldgw=16), **k})
    fwd = lambda l, x=P16, w=P16, b=None, r=None, y=P16, z=None, ws=None, n=0: mqc.mqc_linear_fwd(  # noqa: E731
        l, x, w, b, r, y, z, ws, n, None)
    assert fwd(lin(M=0)) == 0                       # nothing to write
    assert fwd(lin(M=-1)) == -1 and fwd(lin(N=0)) == -1 and fwd(lin(K=0)) == -1
    assert fwd(lin(M=(1 << 30) + 1)) == -1 and fwd(lin(N=(1 << 29) + 1, ldy=1 << 30)) == -1
    assert fwd(lin(K=(1 << 29) + 1, ldx=1 << 30, ldw=1 << 30)) == -1
    assert fwd(lin(act=4)) == -1 and fwd(lin(act=-1)) == -1
    assert fwd(lin(dtype=0)) == -2 and fwd(lin(dtype=3)) == -1
    assert "fp32" in (fwd(lin(dtype=0)), mqc.lib.mqc_last_error_message().decode())[1]
    assert fwd(lin(), x=None) == -1 and fwd(lin(), w=None) == -1 and fwd(lin(), y=None) == -1
    for k in ("x", "w", "y", "z", "r", "b"):
        assert fwd(lin(), **{k: ODD}) == -5, k
    assert fwd(lin(ldx=15)) == -1 and fwd(lin(ldw=8)) == -1 and fwd(lin(ldy=7)) == -1
    assert fwd(lin(ldr=7), r=P16) == -1 and fwd(lin(ldz=0), z=P16) == -1
    many = dict(M=16, ldx=17)                       # rows of 34 bytes: a padded copy is needed
    assert fwd(lin(**many)) == -6
    assert mqc.mqc_linear_fwd_workspace_bytes(lin(M=16)) == 0
    assert mqc.mqc_linear_fwd_workspace_bytes(lin(**many)) == 512
    assert mqc.mqc_linear_fwd_workspace_bytes(lin(ldx=17)) == 0     # few tokens are read as they are
    assert fwd(lin(**many), ws=ODD, n=512) == -5
    bwd = lambda l, g=P16, z=P16, x=P16, w=P16, gx=P16, gw=P16, gb=P16, ws=None, n=0: mqc.mqc_linear_bwd(  # noqa: E731
        l, g, z, x, w, gx, gw, gb, ws, n, None)
    assert bwd(lin()) == -6 and bwd(lin(act=2)) == -6
    assert bwd(lin(), g=None) == -1 and bwd(lin(act=2), z=None) == -1
    assert bwd(lin(), x=None) == -1 and bwd(lin(), w=None) == -1
    for k in ("g", "x", "w", "gx", "gw", "gb"):
        assert bwd(lin(), **{k: ODD}) == -5, k
    assert bwd(lin(ldg=4)) == -1 and bwd(lin(ldgx=4)) == -1 and bwd(lin(ldgw=4)) == -1
    assert bwd(lin(dtype=0)) == -2
    need = mqc.mqc_linear_bwd_workspace_bytes(lin(act=2))
    assert need >= 4 * 8 * 2 and bwd(lin(act=2), ws=P16, n=need - 1) == -6
    assert bwd(lin(M=0), gw=None, gb=None) == 0


def test_group_norm_refusals(mqc):
    d = lambda n=2, c=8, h=3, w=5, s=None: mqc.T4(n, c, h, w, *(s or (h * w * c, 1, w * c, c)))  # noqa: E731

    def fwd(xd=None, yd=None, x=P16, y=P16, dtype=1, groups=4, eps=1e-5, a=0, mean=P16, rstd=P16, ws=P16, n=1 << 20):
        return mqc.mqc_group_norm_fwd(x, xd or d(), dtype, None, None, groups, eps, a, y, yd or xd or d(), mean, rstd,
                                      ws, n, None)
    assert fwd(d(n=0)) == 0
    assert fwd(d(c=0)) == -1 and fwd(d(h=0)) == -1 and fwd(d(w=0)) == -1 and fwd(d(n=-1)) == -1
    assert fwd(groups=3) == -1 and fwd(groups=0) == -1 and fwd(eps=-1.0) == -1 and fwd(eps=float("nan")) == -1
    assert fwd(a=4) == -1 and fwd(dtype=3) == -1
    assert fwd(x=None) == -1 and fwd(y=None) == -1 and fwd(mean=None) == -1 and fwd(rstd=None) == -1
    assert fwd(x=ODD) == -5 and fwd(y=ODD) == -5
    assert fwd(yd=d(c=4)) == -1
    nchw = (120, 15, 5, 1)
    assert fwd(d(s=nchw)) == -2 and "channels last" in mqc.lib.mqc_last_error_message().decode()
    assert fwd(yd=d(s=nchw)) == -2
    assert fwd(d(s=(120, 1, 80, 8))) == -2           # a gap between rows of pixels
    assert fwd(d(s=(120, 1, 20, 4))) == -2           # overlapping pixels
    assert mqc.mqc_group_norm_fwd_workspace_bytes(d(), d(), 1, 4) == 0      # on chip
    wide = lambda n=2: d(n, 32, 400, 400)   # noqa: E731  (1.28 M elements a chunk of eight channels: beyond a cluster)
    need = mqc.mqc_group_norm_fwd_workspace_bytes(wide(), wide(), 0, 4)
    assert need > 0 and fwd(wide(), dtype=0, n=need - 1) == -6 and fwd(wide(), dtype=0, ws=None) == -6
    assert fwd(wide(), dtype=0, ws=ODD) == -5
    need = mqc.mqc_group_norm_bwd_workspace_bytes(d(), d(), d(), 1, 4)
    assert need > 0

    assert fwd(yd=d(s=(0, 1, 40, 8))) == -2 and "overlap" in mqc.lib.mqc_last_error_message().decode()
    assert fwd(yd=d(s=(112, 1, 40, 8))) == -2        # an image ends inside the next
    assert fwd(mean=ctypes.c_void_p(258)) == -5 and fwd(rstd=ctypes.c_void_p(257)) == -5

    def bwd(gd=None, g=P16, x=P16, gx=P16, mean=P16, rstd=P16, groups=4, a=0, ws=P16, n=1 << 20):
        return mqc.mqc_group_norm_bwd(g, gd or d(), x, d(), 1, None, None, mean, rstd, groups, a, gx, d(), P16, P16,
                                      ws, n, None)
    assert bwd(g=None) == -1 and bwd(x=None) == -1 and bwd(gx=None) == -1 and bwd(mean=None) == -1
    assert bwd(gd=d(w=4)) == -1 and bwd(gd=d(s=nchw)) == -2 and bwd(groups=5) == -1 and bwd(a=7) == -1
    assert bwd(g=ODD) == -5 and bwd(n=need - 1) == -6


def test_dropout_refusals(mqc):
    fwd = lambda x=P16, ldx=8, r=None, ldr=0, rows=4, cols=8, dtype=1, p=0.5, dev=None, y=P16, ldy=8: (  # noqa: E731
        mqc.mqc_dropout_fwd(x, ldx, r, ldr, rows, cols, dtype, p, 1, 0, dev, y, ldy, None))
    assert fwd(rows=0) == 0 and fwd(cols=0) == 0
    assert fwd(rows=-1) == -1 and fwd(cols=-1) == -1 and fwd(dtype=3) == -1
    assert fwd(p=-0.1) == -1 and fwd(p=1.1) == -1 and fwd(p=float("nan")) == -1
    assert fwd(x=None) == -1 and fwd(y=None) == -1
    assert fwd(ldx=7) == -1 and fwd(ldy=7) == -1 and fwd(r=P16, ldr=7) == -1
    assert fwd(x=ODD) == -5 and fwd(y=ODD) == -5 and fwd(r=ODD, ldr=8) == -5 and fwd(dev=ODD) == -5
    assert fwd(ldx=16) == -1                          # in place with another row stride
    assert fwd(rows=1 << 40, cols=1 << 40, ldx=1 << 40, ldy=1 << 40) == -1
    bwd = lambda **k: mqc.mqc_dropout_bwd(*{**dict(g=P16, ldg=8, rows=4, cols=8, dtype=1, p=0.5, seed=1, offset=0,  # noqa: E731
                                                 dev=None, gx=P16, ldgx=8), **k}.values(), None)
    assert bwd(g=None) == -1 and bwd(p=2.0) == -1 and bwd(ldg=4) == -1 and bwd(gx=ODD) == -5


def test_quantized_forward_still_refuses_other_activations(mqc):
    """GELU (code 3) belongs to the dense layers alone."""
    mx, cv = mqc.MX(0, 0, 0), mqc.conv_desc(2, 32, 8, 8, 32, 3, 3, 1, 1)
    assert mqc.mqc_conv2d_fwd_quant(P16, P16, mx, P16, P16, mx, cv, mqc.ACT_GELU, mx, P16, P16, None, None, None, 0,
                                    None) == -1


def test_helpers_refuse_host_tensors_and_wrong_types(mqc):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: mqc.linear_fwd(x, x), lambda: mqc.dropout_fwd(x, 0.5, 1),
                 lambda: mqc.group_norm_fwd(x.view(1, 4, 2, 4), 2)):
        with pytest.raises(ValueError):
            call()


def test_helpers_take_their_first_tensor_by_name(mqc):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: mqc.linear_fwd(x=x, w=x), lambda: mqc.dropout_fwd(x=x, p=0.5, seed=1),
                 lambda: mqc.dropout_bwd(p=0.5, seed=1, g=x)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(TypeError):
        mqc.linear_fwd(w=x)


def test_workspace_of_another_device_or_with_gaps_is_refused(mqc):
    class OnDevice:   # what the check looks at
        device = "cuda:0"

        def get_device(self):
            return 0

    with pytest.raises(ValueError, match="workspace"):
        mqc._scratch(64, OnDevice(), torch.empty(64, dtype=torch.uint8))
    host = torch.empty(128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        mqc._scratch(64, host, host[::2])
    assert mqc._scratch(64, host, host)[2] == 128


def test_warps_meet_before_instructions_that_they_execute_together():
    """Cluster barriers and loads from tensor memory of the .aligned form are
    undefined unless all lanes of a warp arrive together, and callers reach
    them from loops and branches that differ by lane: each wrapper brings the
    lanes together itself."""
    import glob
    import os
    import re
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    files = sorted(glob.glob(os.path.join(here, "im2col_gemm_b200", "csrc", "*.cu*")))
    found = []
    for path in files:
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"asm volatile\(\s*\"(barrier\.cluster\.\S*\.aligned|tcgen05\.ld\.sync\.aligned)", text):
            before = text[:m.start()].rstrip()
            found.append((os.path.basename(path), m.group(1), before.endswith("__syncwarp();")))
    assert len(found) >= 6
    assert all(ok for _, _, ok in found), [f for f in found if not f[2]]


def test_a_second_thread_during_the_first_call(mqc, monkeypatch):
    """The first call looks things up; a second thread whose first call falls
    into that finds all of them or looks them up itself."""
    import threading

    class OnDevice:   # what the wrapper looks at
        is_cuda = True

        def get_device(self):
            return 0

    @mqc._on_device
    def call(t):
        return "ran"

    results = []

    def second():
        try:
            results.append(call(OnDevice()))
        except Exception as e:
            results.append(e)

    def device_count():   # releases the interpreter lock
        if threading.current_thread() is threading.main_thread():
            thread = threading.Thread(target=second)
            thread.start()
            thread.join()
        return 1

    for table in ("_DTYPES", "_CUDA"):
        monkeypatch.setattr(mqc, table, {})
    monkeypatch.setattr(torch.cuda, "device_count", device_count)
    assert call(OnDevice()) == "ran" and results == ["ran"]
