"""Python binding of libmqc, the B200 implementation of the MicroQonv hot path
("MicroQonv: Reshaping Convolution Tensors for Efficient Microscaling in
Training and Inference", arXiv:2609.28358).

Argument marshalling only: every computation runs in the CUDA kernels of
``libmqc.so`` (built from ``csrc/`` for sm_100a).  PyTorch supplies device
memory and the current stream.  There is no fallback: importing this module
fails loudly when the library is missing.

The ``mqc_*`` names mirror the C ABI in ``include/mqc.h`` one to one (raw
pointers, sizes, streams).  The lower-case helpers below them allocate the
output tensors with torch and call the same entry points.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmqc.so")

E4M3, E5M2, E2M1 = 0, 1, 2
A32, B32, SQ32 = 0, 1, 2
ORDER_BA, ORDER_AB = 0, 1
ROLE_X, ROLE_W, ROLE_G = 0, 1, 2

STATUS = {0: "MQC_OK", -1: "MQC_ERR_INVALID", -2: "MQC_ERR_UNSUPPORTED", -3: "MQC_ERR_CUDA",
          -4: "MQC_ERR_DEVICE_TIMEOUT", -5: "MQC_ERR_ALIGNMENT", -6: "MQC_ERR_WORKSPACE"}

# every symbol include/mqc.h declares
EXPORTS = ("mqc_codes_bytes", "mqc_scales_bytes", "mqc_tensor_dims", "mqc_quantize_mx", "mqc_im2col_cbf",
           "mqc_im2col_cbf_scales_bytes", "mqc_im2col_cbf_codes_bytes", "mqc_conv2d_fwd", "mqc_conv2d_bwd_data",
           "mqc_conv2d_bwd_weight", "mqc_conv2d_bwd_weight_workspace_bytes", "mqc_get_device_status",
           "mqc_debug_expire_wait", "mqc_status_string", "mqc_last_error_message", "mqc_version",
           "mqc_conv2d_bwd_weight_noalloc", "mqc_conv2d_fwd_workspace_bytes", "mqc_conv2d_bwd_data_workspace_bytes",
           "mqc_quantize_mx_sr", "mqc_conv2d_fwd_quant", "mqc_quantize_mx_batch", "mqc_quantize_nvfp4",
           "mqc_nvfp4_scales_bytes", "mqc_conv2d_fwd_nvfp4", "mqc_group_norm_fwd", "mqc_group_norm_bwd",
           "mqc_group_norm_fwd_workspace_bytes", "mqc_group_norm_bwd_workspace_bytes", "mqc_linear_fwd", "mqc_linear_fwd_workspace_bytes", "mqc_linear_bwd",
           "mqc_linear_bwd_workspace_bytes", "mqc_dropout_fwd", "mqc_dropout_bwd")
NV_A16, NV_B16, NV_SQ16 = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3
F32, BF16, F16 = 0, 1, 2
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


class MqcError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class T4(ctypes.Structure):
    _fields_ = [("d0", ctypes.c_int32), ("d1", ctypes.c_int32), ("d2", ctypes.c_int32), ("d3", ctypes.c_int32),
                ("s0", ctypes.c_int64), ("s1", ctypes.c_int64), ("s2", ctypes.c_int64), ("s3", ctypes.c_int64)]


class MX(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("block", ctypes.c_int32), ("order", ctypes.c_int32)]


class Conv(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "C", "H", "W", "K", "R", "S", "stride_h", "stride_w",
                                               "pad_h", "pad_w")]


class Linear(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("M", "N", "K", "dtype", "act")]
                + [(n, ctypes.c_int64) for n in ("ldx", "ldw", "ldr", "ldy", "ldz", "ldg", "ldgx", "ldgw")])


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python im2col_gemm_b200/build.py` "
                          "(nvcc, sm_100a); there is no fallback implementation")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    P = ctypes.POINTER
    sig = {
        "mqc_codes_bytes": (i64, [P(MX), i32, i32, i32, i32]),
        "mqc_scales_bytes": (i64, [P(MX), i32, i32, i32, i32]),
        "mqc_tensor_dims": (i32, [i32, P(Conv), P(i32)]),
        "mqc_quantize_mx": (i32, [vp, P(T4), P(MX), vp, vp, vp, vp]),
        "mqc_quantize_mx_sr": (i32, [vp, P(T4), P(MX), vp, vp, vp, ctypes.c_uint64, ctypes.c_uint64, vp]),
        "mqc_quantize_mx_batch": (i32, [i32, P(vp), P(T4), P(MX), P(vp), P(vp), P(vp), vp]),
        "mqc_quantize_nvfp4": (i32, [vp, P(T4), i32, i32, vp, vp, vp, vp, vp]),
        "mqc_nvfp4_scales_bytes": (i64, [i32, i32, i32, i32, i32, i32]),
        "mqc_conv2d_fwd_nvfp4": (i32, [vp, vp, vp, i32, vp, vp, vp, i32, P(Conv), vp, vp]),
        "mqc_im2col_cbf": (i32, [vp, vp, P(Conv), P(MX), vp, vp, vp]),
        "mqc_im2col_cbf_scales_bytes": (i64, [P(Conv), P(MX)]),
        "mqc_im2col_cbf_codes_bytes": (i64, [P(Conv), P(MX)]),
        "mqc_conv2d_fwd": (i32, [vp, vp, P(MX), vp, vp, P(MX), P(Conv), vp, vp, sz, vp]),
        "mqc_conv2d_fwd_workspace_bytes": (sz, [P(Conv), P(MX), P(MX)]),
        "mqc_conv2d_fwd_quant": (i32, [vp, vp, P(MX), vp, vp, P(MX), P(Conv), i32, P(MX), vp, vp, vp, vp, vp, sz,
                                       vp]),
        "mqc_conv2d_bwd_data": (i32, [vp, vp, P(MX), vp, vp, P(MX), P(Conv), vp, vp, sz, vp]),
        "mqc_conv2d_bwd_data_workspace_bytes": (sz, [P(Conv), P(MX), P(MX)]),
        "mqc_conv2d_bwd_weight": (i32, [vp, vp, P(MX), vp, vp, P(MX), P(Conv), vp, vp, sz, vp]),
        "mqc_conv2d_bwd_weight_workspace_bytes": (sz, [P(Conv), P(MX), P(MX)]),
        "mqc_conv2d_bwd_weight_noalloc": (i32, [vp, vp, P(MX), vp, vp, P(MX), P(Conv), vp, vp]),
        "mqc_group_norm_fwd": (i32, [vp, P(T4), i32, vp, vp, i32, ctypes.c_float, i32, vp, P(T4), vp, vp, vp, sz, vp]),
        "mqc_group_norm_bwd": (i32, [vp, P(T4), vp, P(T4), i32, vp, vp, vp, vp, i32, i32, vp, P(T4), vp, vp, vp, sz,
                                     vp]),
        "mqc_group_norm_fwd_workspace_bytes": (sz, [P(T4), P(T4), i32, i32]),
        "mqc_group_norm_bwd_workspace_bytes": (sz, [P(T4), P(T4), P(T4), i32, i32]),
        "mqc_linear_fwd": (i32, [P(Linear), vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "mqc_linear_fwd_workspace_bytes": (sz, [P(Linear)]),
        "mqc_linear_bwd": (i32, [P(Linear), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "mqc_linear_bwd_workspace_bytes": (sz, [P(Linear)]),
        "mqc_dropout_fwd": (i32, [vp, i64, vp, i64, i64, i64, i32, ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64,
                                  vp, vp, i64, vp]),
        "mqc_dropout_bwd": (i32, [vp, i64, i64, i64, i32, ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64, vp, vp,
                                  i64, vp]),
        "mqc_get_device_status": (i32, [vp]),
        "mqc_debug_expire_wait": (i32, [i64, vp]),
        "mqc_status_string": (ctypes.c_char_p, [i32]),
        "mqc_last_error_message": (ctypes.c_char_p, []),
        "mqc_version": (i32, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()


def check(status: int) -> None:
    if status != 0:
        raise MqcError(status, lib.mqc_last_error_message().decode())


# ------------------------------------------------------------------ C ABI, same names
def mqc_codes_bytes(mx: MX, d0, d1, d2, d3) -> int:
    return lib.mqc_codes_bytes(ctypes.byref(mx), d0, d1, d2, d3)


def mqc_scales_bytes(mx: MX, d0, d1, d2, d3) -> int:
    return lib.mqc_scales_bytes(ctypes.byref(mx), d0, d1, d2, d3)


def mqc_quantize_mx(src_ptr, desc: T4, mx: MX, codes_ptr, scales_ptr, codes_alt_ptr, stream) -> int:
    return lib.mqc_quantize_mx(src_ptr, ctypes.byref(desc), ctypes.byref(mx), codes_ptr, scales_ptr,
                               codes_alt_ptr, stream)


def mqc_quantize_mx_sr(src_ptr, desc: T4, mx: MX, codes_ptr, scales_ptr, codes_alt_ptr, seed, offset, stream) -> int:
    return lib.mqc_quantize_mx_sr(src_ptr, ctypes.byref(desc), ctypes.byref(mx), codes_ptr, scales_ptr,
                                  codes_alt_ptr, seed, offset, stream)


def mqc_quantize_mx_batch(srcs, descs, mx: MX, codes, scales, codes_alt, stream) -> int:
    """One launch for len(srcs) tensors; pointer lists (ints or c_void_p),
    T4 descriptors, one shared MX; codes_alt a list or None."""
    n = len(srcs)
    arr = lambda xs: (ctypes.c_void_p * n)(*[x.value if isinstance(x, ctypes.c_void_p) else x for x in xs])
    alt = arr(codes_alt) if codes_alt is not None else None
    return lib.mqc_quantize_mx_batch(n, arr(srcs), (T4 * n)(*descs), ctypes.byref(mx), arr(codes), arr(scales),
                                     alt, stream)


def mqc_im2col_cbf(codes_ptr, scales_ptr, conv: Conv, mx: MX, codes_out_ptr, scales_out_ptr, stream) -> int:
    return lib.mqc_im2col_cbf(codes_ptr, scales_ptr, ctypes.byref(conv), ctypes.byref(mx), codes_out_ptr,
                              scales_out_ptr, stream)


def mqc_conv2d_fwd(xq, xs, xf: MX, wq, ws, wf: MX, conv: Conv, y, workspace, workspace_bytes, stream) -> int:
    return lib.mqc_conv2d_fwd(xq, xs, ctypes.byref(xf), wq, ws, ctypes.byref(wf), ctypes.byref(conv), y, workspace,
                              workspace_bytes, stream)


def mqc_conv2d_fwd_quant(xq, xs, xf: MX, wq, ws, wf: MX, conv: Conv, act: int, yf: MX, yq, ys, yq_alt, y, workspace,
                         workspace_bytes, stream) -> int:
    return lib.mqc_conv2d_fwd_quant(xq, xs, ctypes.byref(xf), wq, ws, ctypes.byref(wf), ctypes.byref(conv), act,
                                    ctypes.byref(yf), yq, ys, yq_alt, y, workspace, workspace_bytes, stream)


def mqc_conv2d_fwd_workspace_bytes(conv: Conv, xf: MX, wf: MX) -> int:
    return lib.mqc_conv2d_fwd_workspace_bytes(ctypes.byref(conv), ctypes.byref(xf), ctypes.byref(wf))


def mqc_conv2d_bwd_data(wq, ws, wf: MX, gq, gs, gf: MX, conv: Conv, gx, workspace, workspace_bytes, stream) -> int:
    return lib.mqc_conv2d_bwd_data(wq, ws, ctypes.byref(wf), gq, gs, ctypes.byref(gf), ctypes.byref(conv), gx,
                                   workspace, workspace_bytes, stream)


def mqc_conv2d_bwd_data_workspace_bytes(conv: Conv, wf: MX, gf: MX) -> int:
    return lib.mqc_conv2d_bwd_data_workspace_bytes(ctypes.byref(conv), ctypes.byref(wf), ctypes.byref(gf))


def mqc_conv2d_bwd_weight(gq, gs, gf: MX, xq, xs, xf: MX, conv: Conv, gw, workspace, workspace_bytes,
                          stream) -> int:
    return lib.mqc_conv2d_bwd_weight(gq, gs, ctypes.byref(gf), xq, xs, ctypes.byref(xf), ctypes.byref(conv),
                                     gw, workspace, workspace_bytes, stream)


def mqc_conv2d_bwd_weight_workspace_bytes(conv: Conv, gf: MX, xf: MX) -> int:
    return lib.mqc_conv2d_bwd_weight_workspace_bytes(ctypes.byref(conv), ctypes.byref(gf), ctypes.byref(xf))


def mqc_conv2d_bwd_weight_noalloc(gq, gs, gf: MX, xq, xs, xf: MX, conv: Conv, gw, stream) -> int:
    """Weight gradient with the library's static split-K scratch: no workspace
    argument and no allocation (see include/mqc.h)."""
    return lib.mqc_conv2d_bwd_weight_noalloc(gq, gs, ctypes.byref(gf), xq, xs, ctypes.byref(xf),
                                             ctypes.byref(conv), gw, stream)


def mqc_group_norm_fwd(x, xd: T4, dtype: int, gamma, beta, groups: int, eps: float, act: int, y, yd: T4, mean, rstd,
                       workspace, workspace_bytes, stream) -> int:
    return lib.mqc_group_norm_fwd(x, ctypes.byref(xd), dtype, gamma, beta, groups, eps, act, y, ctypes.byref(yd), mean,
                                  rstd, workspace, workspace_bytes, stream)


def mqc_group_norm_bwd(g, gd: T4, x, xd: T4, dtype: int, gamma, beta, mean, rstd, groups: int, act: int, gx, gxd: T4,
                       ggamma, gbeta, workspace, workspace_bytes, stream) -> int:
    return lib.mqc_group_norm_bwd(g, ctypes.byref(gd), x, ctypes.byref(xd), dtype, gamma, beta, mean, rstd, groups,
                                  act, gx, ctypes.byref(gxd), ggamma, gbeta, workspace, workspace_bytes, stream)


def mqc_group_norm_fwd_workspace_bytes(xd: T4, yd: T4, dtype: int, groups: int) -> int:
    return lib.mqc_group_norm_fwd_workspace_bytes(ctypes.byref(xd), ctypes.byref(yd), dtype, groups)


def mqc_group_norm_bwd_workspace_bytes(gd: T4, xd: T4, gxd: T4, dtype: int, groups: int) -> int:
    return lib.mqc_group_norm_bwd_workspace_bytes(ctypes.byref(gd), ctypes.byref(xd), ctypes.byref(gxd), dtype,
                                                  groups)


def mqc_linear_fwd(lin: Linear, x, w, bias, residual, y, z, workspace, workspace_bytes, stream) -> int:
    return lib.mqc_linear_fwd(ctypes.byref(lin), x, w, bias, residual, y, z, workspace, workspace_bytes, stream)


def mqc_linear_fwd_workspace_bytes(lin: Linear) -> int:
    return lib.mqc_linear_fwd_workspace_bytes(ctypes.byref(lin))


def mqc_linear_bwd(lin: Linear, g, z, x, w, gx, gw, gb, workspace, workspace_bytes, stream) -> int:
    return lib.mqc_linear_bwd(ctypes.byref(lin), g, z, x, w, gx, gw, gb, workspace, workspace_bytes, stream)


def mqc_linear_bwd_workspace_bytes(lin: Linear) -> int:
    return lib.mqc_linear_bwd_workspace_bytes(ctypes.byref(lin))


def mqc_dropout_fwd(x, ldx: int, residual, ldr: int, rows: int, cols: int, dtype: int, p: float, seed: int, offset: int,
                    offset_dev, y, ldy: int, stream) -> int:
    return lib.mqc_dropout_fwd(x, ldx, residual, ldr, rows, cols, dtype, p, seed, offset, offset_dev, y, ldy, stream)


def mqc_dropout_bwd(g, ldg: int, rows: int, cols: int, dtype: int, p: float, seed: int, offset: int, offset_dev, gx,
                    ldgx: int, stream) -> int:
    return lib.mqc_dropout_bwd(g, ldg, rows, cols, dtype, p, seed, offset, offset_dev, gx, ldgx, stream)


def mqc_get_device_status(stream) -> int:
    return lib.mqc_get_device_status(stream)


def mqc_debug_expire_wait(limit_ns: int, stream) -> int:
    return lib.mqc_debug_expire_wait(limit_ns, stream)


# ------------------------------------------------------------------ torch helpers
_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream():
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def conv_desc(N, C, H, W, K, R, S, stride=1, pad=0) -> Conv:
    sh, sw = (stride, stride) if isinstance(stride, int) else stride
    ph, pw = (pad, pad) if isinstance(pad, int) else pad
    return Conv(N, C, H, W, K, R, S, sh, sw, ph, pw)


def conv_out_hw(cv: Conv) -> tuple[int, int]:
    return ((cv.H + 2 * cv.pad_h - cv.R) // cv.stride_h + 1, (cv.W + 2 * cv.pad_w - cv.S) // cv.stride_w + 1)


def tensor_dims(role: int, cv: Conv) -> tuple[int, int, int, int]:
    d = (ctypes.c_int32 * 4)()
    check(lib.mqc_tensor_dims(role, ctypes.byref(cv), d))
    return tuple(d)


class Quantized:
    """Codes + scales of one tensor (device uint8 buffers) and how they are laid out."""

    def __init__(self, codes, scales, dims, mx: MX, codes_alt=None):
        self.codes, self.scales, self.dims, self.mx, self.codes_alt = codes, scales, tuple(dims), mx, codes_alt

    def other_order(self) -> "Quantized":
        """View of the second code order written by the same quantization."""
        if self.codes_alt is None:
            raise ValueError("quantized without the second code order")
        return Quantized(self.codes_alt, self.scales, self.dims, MX(self.mx.fmt, self.mx.block, 1 - self.mx.order),
                         self.codes)


def quantize_mx(src, fmt: int, block: int, order: int, both_orders: bool = False, sr_seed: int | None = None,
                sr_offset: int = 0) -> Quantized:
    """MX-quantize a 4-D fp32 CUDA tensor [d0=B][d1=A][d2][d3] (any strides);
    with `sr_seed`, the elements are rounded stochastically
    (mqc_quantize_mx_sr, order BA, NCHW-like source)."""
    torch = _torch()
    assert src.is_cuda and src.dtype == torch.float32 and src.dim() == 4
    d0, d1, d2, d3 = src.shape
    mx = MX(fmt, block, order)
    nc = mqc_codes_bytes(mx, d0, d1, d2, d3)
    ns = mqc_scales_bytes(mx, d0, d1, d2, d3)
    if nc < 0 or ns < 0:
        raise MqcError(-1, "bad quantization descriptor")
    codes = torch.empty(nc, dtype=torch.uint8, device=src.device)
    scales = torch.empty(ns, dtype=torch.uint8, device=src.device)
    alt = None
    if both_orders:
        alt = torch.empty(mqc_codes_bytes(MX(fmt, block, 1 - order), d0, d1, d2, d3), dtype=torch.uint8,
                          device=src.device)
    desc = T4(d0, d1, d2, d3, *src.stride())
    if sr_seed is None:
        check(mqc_quantize_mx(_ptr(src), desc, mx, _ptr(codes), _ptr(scales), _ptr(alt), _stream()))
    else:
        check(mqc_quantize_mx_sr(_ptr(src), desc, mx, _ptr(codes), _ptr(scales), _ptr(alt), sr_seed, sr_offset,
                                 _stream()))
    return Quantized(codes, scales, (d0, d1, d2, d3), mx, alt)


def quantize_mx_batch(srcs, fmt: int, block: int, order: int, both_orders: bool = False) -> list:
    """MX-quantize several 4-D fp32 CUDA tensors in one launch (same format,
    block mode and order): one Quantized per tensor."""
    torch = _torch()
    mx = MX(fmt, block, order)
    outs = []
    for src in srcs:
        assert src.is_cuda and src.dtype == torch.float32 and src.dim() == 4
        d = tuple(src.shape)
        codes = torch.empty(mqc_codes_bytes(mx, *d), dtype=torch.uint8, device=src.device)
        scales = torch.empty(mqc_scales_bytes(mx, *d), dtype=torch.uint8, device=src.device)
        alt = (torch.empty(mqc_codes_bytes(MX(fmt, block, 1 - order), *d), dtype=torch.uint8, device=src.device)
               if both_orders else None)
        outs.append(Quantized(codes, scales, d, mx, alt))
    descs = [T4(*s.shape, *s.stride()) for s in srcs]
    check(mqc_quantize_mx_batch([s.data_ptr() for s in srcs], descs, mx, [q.codes.data_ptr() for q in outs],
                                [q.scales.data_ptr() for q in outs],
                                [q.codes_alt.data_ptr() for q in outs] if both_orders else None, _stream()))
    return outs


class QuantizedNV(Quantized):
    """NVFP4 codes + E4M3 block scales + the per-tensor fp32 scale (a 2-float
    device buffer: [0] T, [1] scratch)."""

    def __init__(self, codes, scales, dims, block, order, tscale, codes_alt=None):
        super().__init__(codes, scales, dims, MX(E2M1, block, order), codes_alt)
        self.nv_block, self.tscale = block, tscale

    def other_order(self) -> "QuantizedNV":
        if self.codes_alt is None:
            raise ValueError("quantized without the second code order")
        return QuantizedNV(self.codes_alt, self.scales, self.dims, self.nv_block, 1 - self.mx.order, self.tscale,
                           self.codes)


def quantize_nvfp4(src, block: int, order: int, both_orders: bool = False) -> QuantizedNV:
    """NVFP4-quantize a 4-D fp32 CUDA tensor [d0=B][d1=A][d2][d3] (NCHW-like)."""
    torch = _torch()
    assert src.is_cuda and src.dtype == torch.float32 and src.dim() == 4
    d = tuple(src.shape)
    codes = torch.empty(mqc_codes_bytes(MX(E2M1, 0, order), *d), dtype=torch.uint8, device=src.device)
    scales = torch.empty(lib.mqc_nvfp4_scales_bytes(block, order, *d), dtype=torch.uint8, device=src.device)
    alt = (torch.empty(mqc_codes_bytes(MX(E2M1, 0, 1 - order), *d), dtype=torch.uint8, device=src.device)
           if both_orders else None)
    ts = torch.zeros(2, dtype=torch.float32, device=src.device)
    check(lib.mqc_quantize_nvfp4(_ptr(src), ctypes.byref(T4(*d, *src.stride())), block, order, _ptr(codes),
                                 _ptr(scales), _ptr(alt), _ptr(ts), _stream()))
    return QuantizedNV(codes, scales, d, block, order, ts, alt)


def conv2d_fwd_nvfp4(xq: QuantizedNV, wq: QuantizedNV, cv: Conv, out=None):
    """Forward convolution of NVFP4 operands on the tensor core (kind::mxf4nvf4)."""
    torch = _torch()
    P, Q = conv_out_hw(cv)
    y = out if out is not None else torch.empty((cv.N, cv.K, P, Q), dtype=torch.float32, device=xq.codes.device)
    check(lib.mqc_conv2d_fwd_nvfp4(_ptr(xq.codes), _ptr(xq.scales), _ptr(xq.tscale), xq.nv_block, _ptr(wq.codes),
                                   _ptr(wq.scales), _ptr(wq.tscale), wq.nv_block, ctypes.byref(cv), _ptr(y),
                                   _stream()))
    return y


def im2col_cbf(xq: Quantized, cv: Conv):
    """Explicit channel-batch-first im2col of quantized X: (codes, scales)."""
    torch = _torch()
    nc = lib.mqc_im2col_cbf_codes_bytes(ctypes.byref(cv), ctypes.byref(xq.mx))
    ns = lib.mqc_im2col_cbf_scales_bytes(ctypes.byref(cv), ctypes.byref(xq.mx))
    if nc < 0 or ns < 0:
        raise MqcError(-1, "bad im2col descriptor")
    co = torch.empty(nc, dtype=torch.uint8, device=xq.codes.device)
    so = torch.empty(ns, dtype=torch.uint8, device=xq.codes.device)
    check(mqc_im2col_cbf(_ptr(xq.codes), _ptr(xq.scales), cv, xq.mx, _ptr(co), _ptr(so), _stream()))
    return co, so


def conv2d_fwd(xq: Quantized, wq: Quantized, cv: Conv, out=None, workspace=None):
    torch = _torch()
    P, Q = conv_out_hw(cv)
    y = out if out is not None else torch.empty((cv.N, cv.K, P, Q), dtype=torch.float32, device=xq.codes.device)
    nws = mqc_conv2d_fwd_workspace_bytes(cv, xq.mx, wq.mx)
    if workspace is None and nws > 0:
        workspace = torch.empty(nws, dtype=torch.uint8, device=xq.codes.device)
    check(mqc_conv2d_fwd(_ptr(xq.codes), _ptr(xq.scales), xq.mx, _ptr(wq.codes), _ptr(wq.scales), wq.mx, cv,
                         _ptr(y), _ptr(workspace), nws, _stream()))
    return y


def conv2d_fwd_quant(xq: Quantized, wq: Quantized, cv: Conv, fmt: int, block: int, act: int = ACT_NONE,
                     both_orders: bool = False, keep_fp32: bool = False, workspace=None):
    """Forward convolution whose output is returned MX-quantized (order BA,
    and AB with `both_orders`) as the next layer's input: (Quantized, y)
    where y is the fp32 activated output when `keep_fp32`, else None."""
    torch = _torch()
    P, Q = conv_out_hw(cv)
    dev = xq.codes.device
    mx = MX(fmt, block, ORDER_BA)
    dims = (cv.N, cv.K, P, Q)
    codes = torch.empty(mqc_codes_bytes(mx, *dims), dtype=torch.uint8, device=dev)
    scales = torch.empty(mqc_scales_bytes(mx, *dims), dtype=torch.uint8, device=dev)
    alt = (torch.empty(mqc_codes_bytes(MX(fmt, block, ORDER_AB), *dims), dtype=torch.uint8, device=dev)
           if both_orders else None)
    y = torch.empty(dims, dtype=torch.float32, device=dev) if keep_fp32 else None
    nws = mqc_conv2d_fwd_workspace_bytes(cv, xq.mx, wq.mx)
    if workspace is None and nws > 0:
        workspace = torch.empty(nws, dtype=torch.uint8, device=dev)
    check(mqc_conv2d_fwd_quant(_ptr(xq.codes), _ptr(xq.scales), xq.mx, _ptr(wq.codes), _ptr(wq.scales), wq.mx, cv,
                               act, mx, _ptr(codes), _ptr(scales), _ptr(alt), _ptr(y), _ptr(workspace), nws,
                               _stream()))
    return Quantized(codes, scales, dims, mx, alt), y


def conv2d_bwd_data(wq: Quantized, gq: Quantized, cv: Conv, out=None, workspace=None):
    torch = _torch()
    gx = out if out is not None else torch.empty((cv.N, cv.C, cv.H, cv.W), dtype=torch.float32,
                                                 device=gq.codes.device)
    nws = mqc_conv2d_bwd_data_workspace_bytes(cv, wq.mx, gq.mx)
    if workspace is None and nws > 0:
        workspace = torch.empty(nws, dtype=torch.uint8, device=gq.codes.device)
    check(mqc_conv2d_bwd_data(_ptr(wq.codes), _ptr(wq.scales), wq.mx, _ptr(gq.codes), _ptr(gq.scales), gq.mx, cv,
                              _ptr(gx), _ptr(workspace), nws, _stream()))
    return gx


def conv2d_bwd_weight_workspace_bytes(cv: Conv, gf: MX, xf: MX) -> int:
    return mqc_conv2d_bwd_weight_workspace_bytes(cv, gf, xf)


def conv2d_bwd_weight(gq: Quantized, xq: Quantized, cv: Conv, out=None, workspace=None):
    torch = _torch()
    gw = out if out is not None else torch.empty((cv.K, cv.C, cv.R, cv.S), dtype=torch.float32,
                                                 device=gq.codes.device)
    nws = mqc_conv2d_bwd_weight_workspace_bytes(cv, gq.mx, xq.mx)
    if workspace is None and nws > 0:
        workspace = torch.empty(nws, dtype=torch.uint8, device=gq.codes.device)
    check(mqc_conv2d_bwd_weight(_ptr(gq.codes), _ptr(gq.scales), gq.mx, _ptr(xq.codes), _ptr(xq.scales), xq.mx,
                                cv, _ptr(gw), _ptr(workspace), nws, _stream()))
    return gw


# ------------------------------------------------------------------ dense layers
# These calls can be shorter than the host's work around them, so the helpers
# pass plain integers to the library and look up no more than they need.
_DTYPES: dict = {}
_CUDA: dict = {}


def _setup() -> None:
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _CUDA["stream"] = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _CUDA["count"] = torch.cuda.device_count()
    # last, and at once: other threads take it as the sign that all is there
    _DTYPES.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})


def _on_device(fn):
    """Runs fn with its first tensor's device current, so that the launches are
    that device's, and on its current stream (the last argument)."""
    import functools
    first = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, **kwargs):
        t = args[0] if args else kwargs.get(first)
        if t is None:
            raise TypeError(f"{fn.__name__}() needs {first}")
        if not t.is_cuda:
            raise ValueError("the tensors must be on a CUDA device")
        if not _DTYPES:
            _setup()
        device = t.get_device()
        if _CUDA["count"] > 1 and device != _torch().cuda.current_device():
            with _torch().cuda.device(device):
                return fn(*args, **kwargs)
        return fn(*args, **kwargs)

    return call


def _dtype(t) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{t.dtype} tensors are not supported (float32, bfloat16, float16)")
    return code


def _address(t):
    return None if t is None else t.data_ptr()


def _same(first, *others) -> None:
    """The other tensors (None: absent) are on the first one's device, of its type."""
    device, dtype = first.get_device(), first.dtype
    for t in others:
        if t is not None and (t.dtype != dtype or t.get_device() != device):
            raise ValueError(f"expected a {dtype} tensor on {first.device}, got {t.dtype} on {t.device}")


def _params(first, n, *others) -> None:
    """fp32 parameters or statistics of n contiguous elements on the first tensor's device."""
    for t in others:
        if t is not None and (_DTYPES.get(t.dtype) != F32 or t.numel() != n or t.get_device() != first.get_device()
                              or not t.is_contiguous()):
            raise ValueError(f"expected {n} contiguous float32 elements on {first.device}, got {tuple(t.shape)} "
                             f"{t.dtype} on {t.device}")


def _scratch(nbytes: int, like, workspace):
    """(tensor or None, address, bytes): the caller's workspace, or a new one."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = like.new_empty(nbytes, dtype=_torch().uint8)
        return workspace, workspace.data_ptr(), nbytes
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"expected a contiguous workspace on {like.device}, got one on {workspace.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _image_like(x, xd: T4, out) -> tuple:
    """(tensor, descriptor) of an output beside x: `out`, or a new channels-last tensor."""
    if out is not None:
        return out, _image_desc(out, x.shape)
    torch = _torch()
    if x.is_contiguous(memory_format=torch.channels_last):
        return torch.empty_like(x), xd
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device, memory_format=torch.channels_last)
    return y, T4(*x.shape, *y.stride())


def _image_desc(t, shape) -> T4:
    if t.shape != shape:
        raise ValueError(f"expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return T4(*shape, *t.stride())


@_on_device
def group_norm_fwd(x, groups: int, gamma=None, beta=None, eps: float = 1e-5, act: int = ACT_NONE, out=None,
                   workspace=None):
    """act(group norm of x) for a channels-last tensor x [N][C][H][W] (torch's
    channels_last strides, or any pixel and image strides): (y, mean, rstd),
    mean and rstd fp32 [N][groups] for the backward pass."""
    shape, dt = x.shape, _dtype(x)
    if len(shape) != 4:
        raise ValueError("group_norm_fwd takes [N][C][H][W] tensors")
    _same(x, out)
    _params(x, shape[1], gamma, beta)
    xd = _image_desc(x, shape)
    y, yd = _image_like(x, xd, out)
    mean = x.new_empty((shape[0], max(groups, 0)), dtype=_torch().float32)
    rstd = _torch().empty_like(mean)
    ws, at, nws = _scratch(lib.mqc_group_norm_fwd_workspace_bytes(xd, yd, dt, groups), x, workspace)
    check(lib.mqc_group_norm_fwd(x.data_ptr(), xd, dt, _address(gamma), _address(beta), groups, eps, act, y.data_ptr(),
                                 yd, mean.data_ptr(), rstd.data_ptr(), at, nws, _CUDA["stream"](x.get_device())))
    return y, mean, rstd


@_on_device
def group_norm_bwd(g, x, groups: int, mean, rstd, gamma=None, beta=None, act: int = ACT_NONE, out=None,
                   workspace=None):
    """Gradients of group_norm_fwd: (gx, ggamma, gbeta), the last two fp32 [C]."""
    shape, dt = x.shape, _dtype(x)
    if len(shape) != 4:
        raise ValueError("group_norm_bwd takes [N][C][H][W] tensors")
    _same(g, x, out)
    _params(x, shape[1], gamma, beta)
    _params(x, shape[0] * groups, mean, rstd)
    gd, xd = _image_desc(g, shape), _image_desc(x, shape)
    gx, gxd = _image_like(x, xd, out)
    ggamma = x.new_empty(shape[1], dtype=_torch().float32)
    gbeta = _torch().empty_like(ggamma)
    ws, at, nws = _scratch(lib.mqc_group_norm_bwd_workspace_bytes(gd, xd, gxd, dt, groups), x, workspace)
    check(lib.mqc_group_norm_bwd(g.data_ptr(), gd, x.data_ptr(), xd, dt, _address(gamma), _address(beta),
                                 mean.data_ptr(), rstd.data_ptr(), groups, act, gx.data_ptr(), gxd, ggamma.data_ptr(),
                                 gbeta.data_ptr(), at, nws, _CUDA["stream"](x.get_device())))
    return gx, ggamma, gbeta


def _row_stride(t, rows: int, cols: int) -> int:
    """Row stride of a matrix (None: absent) with contiguous rows."""
    if t is None:
        return cols
    if t.shape != (rows, cols):
        raise ValueError(f"expected shape {(rows, cols)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return cols
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError("the elements of a row must be contiguous")
    return row if rows > 1 else max(cols, row)


def _like(t, rows: int, cols: int):
    """A new contiguous matrix of t's shape and type."""
    return _torch().empty_like(t) if t.is_contiguous() else t.new_empty((rows, cols))


def _linear_sizes(name: str, x, w) -> tuple[int, int, int]:
    xs, ws = x.shape, w.shape
    if len(xs) != 2 or len(ws) != 2 or xs[1] != ws[1]:
        raise ValueError(f"{name} takes x [M][K] and w [N][K], got {tuple(xs)} and {tuple(ws)}")
    return xs[0], ws[0], xs[1]


@_on_device
def linear_fwd(x, w, bias=None, act: int = ACT_NONE, residual=None, save_z: bool = False, out=None, workspace=None):
    """(y, z): y = act(x . w^T + bias) + residual for x [M][K] and w [N][K] in
    bf16 or fp16 (rows of any stride), bias fp32 [N]; z, the pre-activation for
    the backward pass, with `save_z`, else None."""
    m, n, k = _linear_sizes("linear_fwd", x, w)
    _same(x, w, residual, out)
    _params(x, n, bias)
    y = out if out is not None else x.new_empty((m, n))
    z = None if not save_z else _torch().empty_like(y) if out is None else x.new_empty((m, n))
    lin = Linear(m, n, k, _dtype(x), act, k if x.is_contiguous() else _row_stride(x, m, k),
                 k if w.is_contiguous() else _row_stride(w, n, k), _row_stride(residual, m, n),
                 _row_stride(out, m, n), n, n, k, k)
    ws, at, nws = _scratch(lib.mqc_linear_fwd_workspace_bytes(lin), x, workspace)
    check(lib.mqc_linear_fwd(lin, x.data_ptr(), w.data_ptr(), _address(bias), _address(residual), y.data_ptr(),
                             _address(z), at, nws, _CUDA["stream"](x.get_device())))
    return y, z


@_on_device
def linear_bwd(g, x, w, z=None, act: int = ACT_NONE, need_x: bool = True, need_w: bool = True, need_bias: bool = True,
               workspace=None):
    """(gx, gw, gb) of linear_fwd for the incoming gradient g [M][N]; z as the
    forward pass saved it (not read for ACT_NONE).  What is not needed is
    None."""
    m, n, k = _linear_sizes("linear_bwd", x, w)
    _same(g, x, w, z)
    gx = _like(x, m, k) if need_x else None
    gw = _like(w, n, k) if need_w else None
    gb = x.new_empty(n, dtype=_torch().float32) if need_bias else None
    lin = Linear(m, n, k, _dtype(x), act, k if x.is_contiguous() else _row_stride(x, m, k),
                 k if w.is_contiguous() else _row_stride(w, n, k), n, n, _row_stride(z, m, n),
                 _row_stride(g, m, n), k, k)
    ws, at, nws = _scratch(lib.mqc_linear_bwd_workspace_bytes(lin), x, workspace)
    check(lib.mqc_linear_bwd(lin, g.data_ptr(), _address(z), x.data_ptr(), w.data_ptr(), _address(gx), _address(gw),
                             _address(gb), at, nws, _CUDA["stream"](g.get_device())))
    return gx, gw, gb


def _dropout_rows(*tensors) -> tuple:
    """(rows, cols, row strides) common to the tensors (None: absent);
    contiguous tensors of any shape are one row."""
    first = tensors[0]
    if all(t is None or t.is_contiguous() for t in tensors):
        n = first.numel()
        return 1, n, (n,) * len(tensors)
    if first.dim() != 2:
        raise ValueError("dropout takes contiguous tensors, or matrices with contiguous rows")
    rows, cols = first.shape
    return rows, cols, tuple(_row_stride(t, rows, cols) for t in tensors)


def _dropout_check(x, other, offset_dev):
    if other is not None and other.shape != x.shape:
        raise ValueError(f"expected shape {tuple(x.shape)}, got {tuple(other.shape)}")
    if offset_dev is not None and (offset_dev.get_device() != x.get_device() or offset_dev.numel() != 1
                                   or offset_dev.dtype != _torch().int64):
        raise ValueError("offset_dev is one int64 element on the tensor's device")


@_on_device
def dropout_fwd(x, p: float, seed: int, offset: int = 0, residual=None, offset_dev=None, out=None):
    """Elements of x dropped with probability p and the others scaled, plus
    `residual`; the random bits depend on (seed, offset) and the element's
    row-major index alone (mqc_dropout_fwd).  `offset_dev`, an int64 CUDA
    tensor of one element, is added to the offset when the kernel runs."""
    _same(x, residual, out)
    _dropout_check(x, residual, offset_dev)
    if out is not None:
        _dropout_check(x, out, None)
    y = out if out is not None else x.new_empty(x.shape)
    rows, cols, (ldx, ldr, ldy) = _dropout_rows(x, residual, y)
    check(lib.mqc_dropout_fwd(x.data_ptr(), ldx, _address(residual), ldr, rows, cols, _dtype(x), p, seed, offset,
                              _address(offset_dev), y.data_ptr(), ldy, _CUDA["stream"](x.get_device())))
    return y


@_on_device
def dropout_bwd(g, p: float, seed: int, offset: int = 0, offset_dev=None, out=None):
    """Gradient of dropout_fwd by x, with the forward call's p, seed and offset."""
    _same(g, out)
    _dropout_check(g, out, offset_dev)
    gx = out if out is not None else g.new_empty(g.shape)
    rows, cols, (ldg, ldgx) = _dropout_rows(g, gx)
    check(lib.mqc_dropout_bwd(g.data_ptr(), ldg, rows, cols, _dtype(g), p, seed, offset, _address(offset_dev),
                              gx.data_ptr(), ldgx, _CUDA["stream"](g.get_device())))
    return gx


def get_device_status() -> int:
    return mqc_get_device_status(_stream())


def debug_expire_wait(limit_ns: int) -> None:
    check(mqc_debug_expire_wait(limit_ns, _stream()))
