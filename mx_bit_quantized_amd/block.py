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

import torch

from . import EPI_NONE, POLICY_BF16, W4A8, _check, lib, mx_scale_shape

# the current stream's handle by device index, without a Stream object (None where this torch has no such call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

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
    if handle is not _bound:  # (a test may load another build)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _bound = handle
    return handle


# The checks below run on every call of operators that may take a few microseconds on the GPU: plain comparisons,
# device indices instead of device objects, the raw stream handle.

def _index(t, name):
    """Device index of a GPU tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    return t.get_device()


def _same(t, name, dev):
    if _index(t, name) != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not on cuda:{dev}")


def _ptr(t, name, dev, dtype, shape):
    """Address of a contiguous tensor of that device, dtype and shape (None for None)."""
    if t is None:
        return None
    _same(t, name, dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (no implicit copies)")
    return t.data_ptr()


def _rows(t, name, dev, shape):
    """(address, row stride) of a bf16 matrix whose rows may be strided."""
    _same(t, name, dev)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must have dtype torch.bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    ld, unit = t.stride()
    if shape[0] > 1 and ld < shape[1] or unit != 1:
        raise ValueError(f"{name} must have unit stride along its rows and rows that do not overlap")
    return t.data_ptr(), (ld if shape[0] > 1 else shape[1])


def _vectors(named, dev, m, n, rows_per_group):
    """Modulation vectors ([n] or [groups, n], rows may be strided) -> (addresses, mod_type, ld_mod, rows_per_group)."""
    ptrs, kind = [], None
    for name, t in named:
        if t is None:
            ptrs.append(None)
            continue
        _same(t, name, dev)
        if t.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
        shape, stride = t.shape, t.stride()
        if not 1 <= len(shape) <= 2 or shape[-1] != n or (n > 1 and stride[-1] != 1) or shape[0] < 1:
            raise ValueError(f"{name} must be [{n}] or [groups, {n}] with unit stride along {n}, got {tuple(shape)}")
        groups = shape[0] if len(shape) == 2 else 1
        this = (t.dtype, groups, stride[0] if groups > 1 else n)
        if kind is None:
            kind = this
        elif kind != this:
            raise ValueError(f"modulation vectors must share dtype, groups and row stride: {name} has {this}, not {kind}")
        ptrs.append(t.data_ptr())
    if kind is None:
        return ptrs, 0, n, 0
    dtype, groups, ld = kind
    if groups == 1 and (rows_per_group is None or rows_per_group >= m):
        rows_per_group = 0
    elif rows_per_group is None or rows_per_group < 1:
        raise ValueError(f"modulation vectors of {groups} groups need rows_per_group")
    elif groups * rows_per_group < m:
        raise ValueError(f"{groups} groups of {rows_per_group} rows do not cover {m} rows")
    return ptrs, (0 if dtype == torch.float32 else 1), ld, rows_per_group


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """(stream handle, context in which to allocate and launch) for work on device ``dev``."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
        return stream.cuda_stream, torch.cuda.stream(stream)  # (sets the device too)
    handle = torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None else _raw_stream(dev)
    return handle, (_HERE if dev == torch.cuda.current_device() else torch.cuda.device(dev))


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D [rows, K]")
    return t.shape


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
    dev = _index(x, "x")
    m, k = _matrix(x, "x")
    if h is not None and (branch is None or not write_h):
        raise ValueError("h is an output of a call with a branch and write_h")
    if out_scales is not None and mode == POLICY_BF16:
        raise ValueError("POLICY_BF16 has no out_scales")
    bf16, u8 = torch.bfloat16, torch.uint8
    px, ldx = _rows(x, "x", dev, (m, k))
    if gate is None and scale is None and shift is None:
        pg = psc = psh = None
        mod_type, ld_mod, rpg = 0, k, 0
    else:
        (pg, psc, psh), mod_type, ld_mod, rpg = _vectors((("gate", gate), ("scale", scale), ("shift", shift)), dev, m, k,
                                                         rows_per_group)
    vec = (k,)
    ppw, ppb = _ptr(post_weight, "post_weight", dev, bf16, vec), _ptr(post_bias, "post_bias", dev, bf16, vec)
    pw, pbias = _ptr(weight, "weight", dev, bf16, vec), _ptr(bias, "bias", dev, bf16, vec)
    pm = _ptr(act_mult, "act_mult", dev, torch.float32, vec)
    handle, ctx = _on(dev, stream)
    with ctx:
        pb = ph = None
        ldb = ldh = k
        if branch is not None:
            pb, ldb = _rows(branch, "branch", dev, (m, k))
            if write_h:
                if h is None:
                    h = torch.empty_like(x) if ldx == k else torch.empty((m, k), dtype=bf16, device=x.device)
                    ph = h.data_ptr()
                else:
                    ph, ldh = _rows(h, "h", dev, (m, k))
            else:
                h = None
        elif write_h:
            h = x
        pos = None
        if mode == POLICY_BF16:
            if out is None:
                out = torch.empty_like(x) if ldx == k else torch.empty((m, k), dtype=bf16, device=x.device)
                po = out.data_ptr()
            else:
                po = _ptr(out, "out", dev, bf16, (m, k))
        else:
            wide = mode == W4A8
            codes_shape = (m, k if wide else k // 2)
            scales_shape, scales_type = ((m,), torch.float32) if wide else (mx_scale_shape(m, k), u8)
            if out is None:
                out = torch.empty(codes_shape, dtype=u8, device=x.device)
                po = out.data_ptr()
            else:
                po = _ptr(out, "out", dev, u8, codes_shape)
            if out_scales is None:
                out_scales = torch.empty(scales_shape, dtype=scales_type, device=x.device)
                pos = out_scales.data_ptr()
            else:
                pos = _ptr(out_scales, "out_scales", dev, scales_type, scales_shape)
        args = NormArgs(px, pb, pg, ppw, ppb, pw, pbias, psc, psh, pm, ph, po, pos, m, k, ldx, ldb, ldh, ld_mod, rpg,
                        post_norm, norm, mod_type, eps, branch_scale)
        st = _lib().mxq_norm_quantize(mode, args, handle)
    _check(st, "norm_quantize")
    return out, out_scales, h


def _operands(mode, a_codes, a_scales, w_codes, w_scales):
    """Device, (M, weight rows, K) and addresses of a product's quantized operands."""
    dev = _index(w_codes, "w_codes")
    n, half = _matrix(w_codes, "w_codes")
    k = 2 * half
    _same(a_codes, "a_codes", dev)
    m = _matrix(a_codes, "a_codes")[0]
    u8 = torch.uint8
    if mode == W4A8:
        pa = _ptr(a_codes, "a_codes", dev, u8, (m, k))
        ps = _ptr(a_scales, "a_scales", dev, torch.float32, (m,))
    else:
        pa = _ptr(a_codes, "a_codes", dev, u8, (m, half))
        ps = _ptr(a_scales, "a_scales", dev, u8, mx_scale_shape(m, k))
    return dev, m, n, k, pa, ps, _ptr(w_codes, "w_codes", dev, u8, (n, half)), _ptr(w_scales, "w_scales", dev, u8,
                                                                                    mx_scale_shape(n, k))


def gemm_residual(mode, a_codes, a_scales, w_codes, w_scales, residual, bias=None, gate=None, rows_per_group=None,
                  epilogue=EPI_NONE, y=None, stream=None):
    """y = bf16(residual + gate * epilogue(A W^T + bias)): the scaled GEMM into a residual stream.

    residual bf16 [M, N]; ``y`` may be residual itself (in place). gate is [N] or [groups, N], float32 or bfloat16,
    row m using vector m // rows_per_group.
    """
    dev, m, n, k, pa, ps, pw, pws = _operands(mode, a_codes, a_scales, w_codes, w_scales)
    bf16 = torch.bfloat16
    pr = _ptr(residual, "residual", dev, bf16, (m, n))
    pb = _ptr(bias, "bias", dev, bf16, (n,))
    if gate is None:
        pg, mod_type, ld, rpg = None, 0, n, 0
    else:
        (pg,), mod_type, ld, rpg = _vectors((("gate", gate),), dev, m, n, rows_per_group)
    handle, ctx = _on(dev, stream)
    with ctx:
        if y is None:
            y = torch.empty_like(residual)
            py = y.data_ptr()
        else:
            py = _ptr(y, "y", dev, bf16, (m, n))
        st = _lib().mxq_gemm_residual(mode, pa, ps, pw, pws, pb, epilogue, pr, pg, mod_type, ld, rpg, py, m, n, k, handle)
    _check(st, "gemm_residual")
    return y


def quantize_weight_gated_mxfp4(w_gate, w_up, codes=None, scales=None, stream=None):
    """RTN MXFP4 packing of a gated block's two projections, bf16 [H, K] each, for gemm_gated -> (codes, scales).

    codes: uint8 [2H, K/2], the rows of the two weights interleaved by 32; scales: uint8 [ceil(K/128), 2H, 4].
    """
    dev = _index(w_gate, "w_gate")
    h, k = _matrix(w_gate, "w_gate")
    bf16, u8 = torch.bfloat16, torch.uint8
    pg, pu = _ptr(w_gate, "w_gate", dev, bf16, (h, k)), _ptr(w_up, "w_up", dev, bf16, (h, k))
    handle, ctx = _on(dev, stream)
    with ctx:
        if codes is None:
            codes = torch.empty((2 * h, k // 2), dtype=u8, device=w_gate.device)
        if scales is None:
            scales = torch.empty(mx_scale_shape(2 * h, k), dtype=u8, device=w_gate.device)
        st = _lib().mxq_quantize_weight_gated_mxfp4(pg, pu, h, k, k, _ptr(codes, "codes", dev, u8, (2 * h, k // 2)),
                                                    _ptr(scales, "scales", dev, u8, mx_scale_shape(2 * h, k)), handle)
    _check(st, "quantize_weight_gated_mxfp4")
    return codes, scales


def gemm_gated(mode, a_codes, a_scales, w_codes, w_scales, act, bias_gate=None, bias_up=None, mxfp4_out=False, y=None,
               y_scales=None, stream=None):
    """Gated feed-forward block's hidden state, act(A Wg^T + bias_gate) * (A Wu^T + bias_up).

    w_codes, w_scales from quantize_weight_gated_mxfp4. bf16 [M, H] by default; with ``mxfp4_out`` (W4A4; or y_scales
    given) the second projection's MXFP4 activation, (codes, scales), as quantize_act makes it of the bf16 hidden state.
    """
    dev, m, n, k, pa, ps, pw, pws = _operands(mode, a_codes, a_scales, w_codes, w_scales)
    if n % 2 != 0:
        raise ValueError("w_codes must hold the rows of both projections (quantize_weight_gated_mxfp4)")
    h = n // 2
    bf16, u8 = torch.bfloat16, torch.uint8
    pg, pu = _ptr(bias_gate, "bias_gate", dev, bf16, (h,)), _ptr(bias_up, "bias_up", dev, bf16, (h,))
    handle, ctx = _on(dev, stream)
    with ctx:
        if mxfp4_out or y_scales is not None:
            mxfp4_out = True
            if y is None:
                y = torch.empty((m, h // 2), dtype=u8, device=a_codes.device)
                py = y.data_ptr()
            else:
                py = _ptr(y, "y", dev, u8, (m, h // 2))
            if y_scales is None:
                y_scales = torch.empty(mx_scale_shape(m, h), dtype=u8, device=a_codes.device)
                pys = y_scales.data_ptr()
            else:
                pys = _ptr(y_scales, "y_scales", dev, u8, mx_scale_shape(m, h))
        else:
            pys = None
            if y is None:
                y = torch.empty((m, h), dtype=bf16, device=a_codes.device)
                py = y.data_ptr()
            else:
                py = _ptr(y, "y", dev, bf16, (m, h))
        st = _lib().mxq_gemm_gated(mode, pa, ps, pw, pws, pg, pu, act, py, pys, m, h, k, handle)
    _check(st, "gemm_gated")
    return (y, y_scales) if mxfp4_out else y


def block_kernel_name(mode, M, N, K, gated=False, mxfp4_out=False):
    """Name of the kernel that gemm_residual (or with ``gated`` gemm_gated, N = H) runs for a shape (host query).

    By the shape alone: gemm_residual with a gate of several groups whose row stride is no multiple of 8 runs the split-K one.
    """
    return _lib().mxq_block_kernel_name(int(mode), int(gated), int(mxfp4_out), int(M), int(N), int(K)).decode()
