"""Binding of the operators around the quantized linears of a transformer block (include/mxq_block.h).

    norm_quantize(mode, x, branch=None, gate=None, ...)       -> (out, scales, h)
    gemm_residual(mode, a_codes, a_scales, w_codes, w_scales, residual, bias=None, gate=None, ...) -> y
    quantize_weight_gated_mxfp4(w_gate, w_up)                 -> (codes, scales)
    gemm_gated(mode, a_codes, a_scales, w_codes, w_scales, act, ...) -> hidden or (codes, scales)
    block_kernel_name(mode, M, N, K, gated=False, mxfp4_out=False)

All tensors of a call live on one device, which need not be the current one; the work goes to
``stream``, or to that device's current stream. Outputs that a call allocates belong to that stream.
Shapes and devices are checked here, sizes and alignment in the library; nothing is copied.
"""

import contextlib
import ctypes

from . import (EPI_NONE, POLICY_BF16, W4A4, W4A8, _check, _torch, lib, mx_scale_shape)

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
GATED_SILU, GATED_GELU_TANH = 0, 1
NORM_MAX_K = 32768  # MXQ_NORM_MAX_K

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_INT = ctypes.c_int


class NormArgs(ctypes.Structure):
    """mxq_norm_args."""
    _fields_ = ([(n, _P) for n in ("x", "branch", "gate", "post_weight", "post_bias", "weight", "bias", "scale", "shift",
                                   "act_mult", "h", "out", "out_scales")]
                + [(n, _I64) for n in ("M", "K", "ldx", "ldb", "ldh", "ld_mod", "rows_per_group")]
                + [(n, _I32) for n in ("post_norm", "norm", "mod_type")]
                + [("eps", ctypes.c_float), ("branch_scale", ctypes.c_float)])


# every function include/mxq_block.h declares, with its ctypes signature
_SIGS = {
    "mxq_norm_quantize": (_INT, [_INT, ctypes.POINTER(NormArgs), _P]),
    "mxq_gemm_residual": (_INT, [_INT, _P, _P, _P, _P, _P, _INT, _P, _P, _INT, _I64, _I64, _P, _I64, _I64, _I64, _P]),
    "mxq_quantize_weight_gated_mxfp4": (_INT, [_P, _P, _I64, _I64, _I64, _P, _P, _P]),
    "mxq_gemm_gated": (_INT, [_INT, _P, _P, _P, _P, _P, _P, _INT, _P, _P, _I64, _I64, _I64, _P]),
    "mxq_block_kernel_name": (ctypes.c_char_p, [_INT, _INT, _INT, _I64, _I64, _I64]),
}

_bound = None


def _lib():
    global _bound
    handle = lib()
    if handle is not _bound:
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _bound = handle
    return handle


def _device(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    return t.device


def _ptr(t, name, device, dtype, shape=None):
    """Address of a contiguous tensor on ``device`` (None for None)."""
    if t is None:
        return None
    if _device(t, name) != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (no implicit copies)")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _rows(t, name, device, shape):
    """(address, row stride) of a bf16 matrix whose rows may be strided."""
    torch = _torch()
    if _device(t, name) != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must have dtype torch.bfloat16, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if shape[0] > 1 and t.stride(0) < shape[1] or shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its rows and rows that do not overlap")
    return t.data_ptr(), (t.stride(0) if shape[0] > 1 else shape[1])


def _vectors(named, device, m, n, rows_per_group):
    """Modulation vectors ([n] or [groups, n], rows may be strided) -> (addresses, mod_type, ld_mod, rows_per_group)."""
    torch = _torch()
    ptrs, kind, ld, groups = [], None, n, 1
    for name, t in named:
        if t is None:
            ptrs.append(None)
            continue
        if _device(t, name) != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")
        if t.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
        v = t if t.dim() == 2 else t.unsqueeze(0)
        if v.dim() != 2 or v.shape[1] != n or (n > 1 and v.stride(1) != 1) or v.shape[0] < 1:
            raise ValueError(f"{name} must be [{n}] or [groups, {n}] with unit stride along {n}, got {tuple(t.shape)}")
        this = (t.dtype, v.shape[0], v.stride(0) if v.shape[0] > 1 else n)
        if kind is None:
            kind = this
        elif kind[:2] != this[:2] or (kind[1] > 1 and kind[2] != this[2]):
            raise ValueError(f"modulation vectors must share dtype, groups and row stride: {name} has {this}, not {kind}")
        ptrs.append(v.data_ptr())
    if kind is None:
        return ptrs, 0, n, 0
    groups, ld = kind[1], kind[2]
    if groups == 1 and (rows_per_group is None or rows_per_group >= m):
        rpg = 0
    elif rows_per_group is None or rows_per_group < 1:
        raise ValueError(f"modulation vectors of {groups} groups need rows_per_group")
    elif groups * rows_per_group < m:
        raise ValueError(f"{groups} groups of {rows_per_group} rows do not cover {m} rows")
    else:
        rpg = int(rows_per_group)
    return ptrs, (0 if kind[0] == torch.float32 else 1), ld, rpg


def _on(device, stream):
    """(stream handle, context in which to allocate and launch) for work on ``device``."""
    torch = _torch()
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return stream.cuda_stream, torch.cuda.stream(stream)  # (sets the device too)
    ctx = contextlib.nullcontext() if device.index == torch.cuda.current_device() else torch.cuda.device(device)
    return torch.cuda.current_stream(device).cuda_stream, ctx


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D [rows, K]")
    return int(t.shape[0]), int(t.shape[1])


def norm_quantize(mode, x, branch=None, gate=None, branch_scale=1.0, post_norm=NORM_NONE, post_weight=None,
                  post_bias=None, norm=NORM_RMS, weight=None, bias=None, scale=None, shift=None, rows_per_group=None,
                  eps=1e-6, act_mult=None, h=None, write_h=True, out=None, out_scales=None, stream=None):
    """Residual add, norm, modulation and the next linear's activation format -> (out, scales, h).

    h = bf16(x + branch_scale * gate * post_norm(branch)), n = norm(h) * weight + bias, then n * (1 + scale) + shift in bf16:
    returned as it is for POLICY_BF16 (scales None), as quantize_act's codes and scales for W4A4 and W4A8, or as
    quantize_mxfp4_hadamard's (with ``act_mult``) for POLICY_TRANSFORM_ON. Without a branch h is x. ``h`` may be x or branch
    (in place); ``write_h=False`` keeps h out of memory. gate, scale and shift are [K] or [groups, K], float32 or bfloat16
    alike, row m using vector m // rows_per_group.
    """
    torch = _torch()
    device = _device(x, "x")
    m, k = _matrix(x, "x")
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    a = NormArgs()
    a.x, a.ldx = _rows(x, "x", device, (m, k))
    (a.gate, a.scale, a.shift), a.mod_type, a.ld_mod, a.rows_per_group = _vectors(
        (("gate", gate), ("scale", scale), ("shift", shift)), device, m, k, rows_per_group)
    for name, t in (("post_weight", post_weight), ("post_bias", post_bias), ("weight", weight), ("bias", bias)):
        if t is not None:
            setattr(a, name, _ptr(t, name, device, bf16, (k,)))
    if act_mult is not None:
        a.act_mult = _ptr(act_mult, "act_mult", device, f32, (k,))
    a.M, a.K = m, k
    a.norm, a.post_norm, a.eps, a.branch_scale = int(norm), int(post_norm), float(eps), float(branch_scale)
    handle, ctx = _on(device, stream)
    with ctx:
        if branch is not None:
            a.branch, a.ldb = _rows(branch, "branch", device, (m, k))
            if write_h:
                if h is None:
                    h = torch.empty((m, k), dtype=bf16, device=device)
                a.h, a.ldh = _rows(h, "h", device, (m, k))
            else:
                h = None
        elif h is None:
            h = x if write_h else None
        else:
            raise ValueError("h is an output of a call with a branch")
        if mode == POLICY_BF16:
            if out is None:
                out = torch.empty((m, k), dtype=bf16, device=device)
            a.out = _ptr(out, "out", device, bf16, (m, k))
        else:
            wide = mode == W4A8
            if out is None:
                out = torch.empty((m, k if wide else k // 2), dtype=u8, device=device)
            if out_scales is None:
                out_scales = torch.empty((m,) if wide else mx_scale_shape(m, k), dtype=f32 if wide else u8, device=device)
            a.out = _ptr(out, "out", device, u8, (m, k if wide else k // 2))
            a.out_scales = _ptr(out_scales, "out_scales", device, f32 if wide else u8,
                                (m,) if wide else mx_scale_shape(m, k))
        st = _lib().mxq_norm_quantize(int(mode), ctypes.byref(a), handle)
    _check(st, "norm_quantize")
    return out, out_scales, h


def _operands(mode, a_codes, a_scales, w_codes, w_scales):
    """Device, (M, weight rows, K) and addresses of a product's quantized operands."""
    torch = _torch()
    device = _device(w_codes, "w_codes")
    n, half = _matrix(w_codes, "w_codes")
    k = 2 * half
    m = int(a_codes.shape[0])
    u8 = torch.uint8
    ptrs = [_ptr(a_codes, "a_codes", device, u8, (m, k if mode == W4A8 else half)),
            _ptr(a_scales, "a_scales", device, torch.float32 if mode == W4A8 else u8,
                 (m,) if mode == W4A8 else mx_scale_shape(m, k)),
            _ptr(w_codes, "w_codes", device, u8, (n, half)), _ptr(w_scales, "w_scales", device, u8, mx_scale_shape(n, k))]
    return device, m, n, k, ptrs


def gemm_residual(mode, a_codes, a_scales, w_codes, w_scales, residual, bias=None, gate=None, rows_per_group=None,
                  epilogue=EPI_NONE, y=None, stream=None):
    """y = bf16(residual + gate * epilogue(A W^T + bias)): the scaled GEMM into a residual stream.

    residual bf16 [M, N]; ``y`` may be residual itself (in place). gate is [N] or [groups, N], float32 or bfloat16,
    row m using vector m // rows_per_group.
    """
    torch = _torch()
    device, m, n, k, ptrs = _operands(mode, a_codes, a_scales, w_codes, w_scales)
    bf16 = torch.bfloat16
    res = _ptr(residual, "residual", device, bf16, (m, n))
    b = _ptr(bias, "bias", device, bf16, (n,))
    (g,), mod_type, ld, rpg = _vectors((("gate", gate),), device, m, n, rows_per_group)
    handle, ctx = _on(device, stream)
    with ctx:
        if y is None:
            y = torch.empty((m, n), dtype=bf16, device=device)
        st = _lib().mxq_gemm_residual(int(mode), *ptrs, b, int(epilogue), res, g, mod_type, ld, rpg,
                                      _ptr(y, "y", device, bf16, (m, n)), m, n, k, handle)
    _check(st, "gemm_residual")
    return y


def quantize_weight_gated_mxfp4(w_gate, w_up, codes=None, scales=None, stream=None):
    """RTN MXFP4 packing of a gated block's two projections, bf16 [H, K] each, for gemm_gated -> (codes, scales).

    codes: uint8 [2H, K/2], the rows of the two weights interleaved by 32; scales: uint8 [ceil(K/128), 2H, 4].
    """
    torch = _torch()
    device = _device(w_gate, "w_gate")
    h, k = _matrix(w_gate, "w_gate")
    bf16, u8 = torch.bfloat16, torch.uint8
    pg, pu = _ptr(w_gate, "w_gate", device, bf16), _ptr(w_up, "w_up", device, bf16, (h, k))
    handle, ctx = _on(device, stream)
    with ctx:
        if codes is None:
            codes = torch.empty((2 * h, k // 2), dtype=u8, device=device)
        if scales is None:
            scales = torch.empty(mx_scale_shape(2 * h, k), dtype=u8, device=device)
        st = _lib().mxq_quantize_weight_gated_mxfp4(pg, pu, h, k, k, _ptr(codes, "codes", device, u8, (2 * h, k // 2)),
                                                    _ptr(scales, "scales", device, u8, mx_scale_shape(2 * h, k)), handle)
    _check(st, "quantize_weight_gated_mxfp4")
    return codes, scales


def gemm_gated(mode, a_codes, a_scales, w_codes, w_scales, act, bias_gate=None, bias_up=None, mxfp4_out=False, y=None,
               y_scales=None, stream=None):
    """Gated feed-forward block's hidden state, act(A Wg^T + bias_gate) * (A Wu^T + bias_up).

    w_codes, w_scales from quantize_weight_gated_mxfp4. bf16 [M, H] by default; with ``mxfp4_out`` (W4A4; or y_scales
    given) the second projection's MXFP4 activation, (codes, scales), as quantize_act makes it of the bf16 hidden state.
    """
    torch = _torch()
    device, m, n, k, ptrs = _operands(mode, a_codes, a_scales, w_codes, w_scales)
    if n % 2 != 0:
        raise ValueError("w_codes must hold the rows of both projections (quantize_weight_gated_mxfp4)")
    h = n // 2
    bf16, u8 = torch.bfloat16, torch.uint8
    bg, bu = _ptr(bias_gate, "bias_gate", device, bf16, (h,)), _ptr(bias_up, "bias_up", device, bf16, (h,))
    mxfp4_out = mxfp4_out or y_scales is not None
    if mxfp4_out and h % 32 != 0:
        raise ValueError("an MXFP4 hidden state needs a multiple of 32 columns")
    handle, ctx = _on(device, stream)
    with ctx:
        if y is None:
            y = torch.empty((m, h // 2), dtype=u8, device=device) if mxfp4_out else \
                torch.empty((m, h), dtype=bf16, device=device)
        if mxfp4_out and y_scales is None:
            y_scales = torch.empty(mx_scale_shape(m, h), dtype=u8, device=device)
        st = _lib().mxq_gemm_gated(int(mode), *ptrs, bg, bu, int(act),
                                   _ptr(y, "y", device, u8 if mxfp4_out else bf16, (m, h // 2 if mxfp4_out else h)),
                                   _ptr(y_scales, "y_scales", device, u8, mx_scale_shape(m, h)), m, h, k, handle)
    _check(st, "gemm_gated")
    return (y, y_scales) if mxfp4_out else y


def block_kernel_name(mode, M, N, K, gated=False, mxfp4_out=False):
    """Name of the kernel that gemm_residual (or with ``gated`` gemm_gated, N = H) runs for a shape (host query)."""
    return _lib().mxq_block_kernel_name(int(mode), int(gated), int(mxfp4_out), int(M), int(N), int(K)).decode()
