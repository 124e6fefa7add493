"""Binding of the attention half of a transformer block (include/mxq_attention.h).

    page_plan(cached, added, block_table, free_pages, page_size, tokens)  -> PagePlan
    rotary_frequencies(pairs_per_axis, theta)                            -> (freqs, axis)
    kv_cache(pages, kv_heads, page_size, head_dim, fmt)                  -> KvCache
    rotary_qkv(qkv, heads, kv_heads, head_dim, positions, freqs, axis, ...) -> (q, k)
    attention(q, k, v, starts_q=None, starts_k=None, ...)                -> out
    attention_paged(q, cache, block_table, lengths, ...)                 -> out

All tensors of a call live on one device, which need not be the current one; the work goes to
``stream``, or to that device's current stream. Outputs and workspaces that a call allocates belong
to that stream. Shapes and devices are checked here, sizes and alignment in the library; nothing is
copied, and nothing that lies on the device (lengths, tables, slots) is read by the host.
"""

import collections
import ctypes
import math

import torch

from . import _check, lib
from . import block
from .block import _index, _on, _rows, _same

KV_BF16, KV_MXFP8 = 0, 1
ROTARY_NORM_NONE, ROTARY_NORM_ROW, ROTARY_NORM_HEAD = 0, 1, 2
MAX_REQUESTS = 4096  # MXQ_MAX_REQUESTS

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_INT = ctypes.c_int
_F32 = ctypes.c_float


class KvCacheArgs(ctypes.Structure):
    """mxq_kv_cache."""
    _fields_ = ([(n, _P) for n in ("k", "v", "k_scales", "v_scales")] + [(n, _I64) for n in ("pages", "page_size")]
                + [(n, _I32) for n in ("kv_heads", "head_dim", "format")])


class RotaryArgs(ctypes.Structure):
    """mxq_rotary_args."""
    _fields_ = ([(n, _P) for n in ("qkv", "positions", "freqs", "axis", "q_weight", "k_weight", "q", "k", "slots")]
                + [(n, _I64) for n in ("M", "ldx", "ldq", "ldk", "ld_pos")]
                + [(n, _I32) for n in ("heads", "kv_heads", "head_dim", "axes", "pairs", "interleaved", "norm")]
                + [("eps", _F32)])


class AttentionArgs(ctypes.Structure):
    """mxq_attention_args."""
    _fields_ = ([(n, _P) for n in ("q", "k", "v", "starts_q", "starts_k", "out")]
                + [(n, _I64) for n in ("sequences", "Mq", "Mk", "ldq", "ldk", "ldv", "ldo", "left", "right", "sinks")]
                + [(n, _I32) for n in ("heads", "kv_heads", "head_dim")] + [("scale", _F32)])


class PagedArgs(ctypes.Structure):
    """mxq_paged_args."""
    _fields_ = ([(n, _P) for n in ("q", "block_table", "lengths", "out")]
                + [(n, _I64) for n in ("sequences", "width", "ldq", "ldo", "left", "sinks")]
                + [("heads", _I32), ("scale", _F32)])


_SIZE = ctypes.POINTER(ctypes.c_size_t)
_CACHE = ctypes.POINTER(KvCacheArgs)
# every function include/mxq_attention.h declares, with its ctypes signature
_SIGS = {
    "mxq_page_plan": (_INT, [_P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P]),
    "mxq_rotary_qkv": (_INT, [ctypes.POINTER(RotaryArgs), _CACHE, _P]),
    "mxq_attention_workspace_bytes": (_INT, [ctypes.POINTER(AttentionArgs), _SIZE]),
    "mxq_attention": (_INT, [ctypes.POINTER(AttentionArgs), _P, ctypes.c_size_t, _P]),
    "mxq_attention_paged_workspace_bytes": (_INT, [ctypes.POINTER(PagedArgs), _CACHE, _SIZE]),
    "mxq_attention_paged": (_INT, [ctypes.POINTER(PagedArgs), _CACHE, _P, ctypes.c_size_t, _P]),
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
    return _bound


#: What page_plan returns, int32 each: slots [tokens] and positions [tokens] (-1 and 0 behind the last token), starts
#: [requests + 1], lengths [requests], taken [2] (pages taken from the list, new tokens without a page).
PagePlan = collections.namedtuple("PagePlan", "slots positions starts lengths taken")

#: A paged cache: k and v [pages, kv_heads, page_size, head_dim], bf16, or uint8 E4M3 codes with scales
#: [pages, kv_heads, page_size, head_dim / 32] (MXFP8).
KvCache = collections.namedtuple("KvCache", "k v k_scales v_scales", defaults=(None, None))


def kv_cache(pages, kv_heads, page_size, head_dim, fmt=KV_BF16, device="cuda"):
    """A cache of zeros."""
    shape = (pages, kv_heads, page_size, head_dim)
    if fmt == KV_BF16:
        return KvCache(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
    if fmt != KV_MXFP8:
        raise ValueError(f"unknown cache format {fmt}")
    return KvCache(*(torch.zeros(s, dtype=torch.uint8, device=device)
                     for s in (shape, shape, shape[:3] + (head_dim // 32,), shape[:3] + (head_dim // 32,))))


def rotary_frequencies(pairs_per_axis, theta=10000.0, device="cuda"):
    """(freqs float64 [pairs], axis int32 [pairs]) of consecutive axes with n pairs each: theta^(-i / n), i < n, per axis."""
    counts = [pairs_per_axis] if isinstance(pairs_per_axis, int) else list(pairs_per_axis)
    freqs = [theta ** (-i / n) for n in counts for i in range(n)]
    axis = [a for a, n in enumerate(counts) for _ in range(n)]
    return (torch.tensor(freqs, dtype=torch.float64, device=device), torch.tensor(axis, dtype=torch.int32, device=device))


def _ptr(t, name, dev, dtype, shape):
    """block._ptr, with the usual case in one comparison."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return block._ptr(t, name, dev, dtype, shape)


def _heads(t, name, dev, rows=None, heads=None, d=None):
    """(address, row stride) of a bf16 [rows, heads, d] tensor: heads side by side, rows that may be strided."""
    _same(t, name, dev)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must have dtype torch.bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or (rows is not None and shape[0] != rows) or (heads is not None and shape[1] != heads) or \
            (d is not None and shape[2] != d):
        want = ", ".join("rows" if n is None and i == 0 else "heads" if n is None else str(n)
                         for i, n in enumerate((rows, heads, d)))
        raise ValueError(f"{name} must have shape [{want}], got {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1] * shape[2]
    ld, sh, se = t.stride()
    if (se != 1 and shape[2] > 1) or (sh != shape[2] and shape[1] > 1) or (shape[0] > 1 and ld < shape[1] * shape[2]):
        raise ValueError(f"{name} must have its heads side by side and rows that do not overlap")
    return t.data_ptr(), (ld if shape[0] > 1 else shape[1] * shape[2])


def _cache_args(cache, dev):
    """mxq_kv_cache of a KvCache."""
    k = cache.k
    _same(k, "cache.k", dev)
    if k.dim() != 4:
        raise ValueError("cache.k must be [pages, kv_heads, page_size, head_dim]")
    shape = k.shape
    pages, heads, page, d = shape
    if cache.k_scales is None and cache.v_scales is None:
        bf16 = torch.bfloat16
        return KvCacheArgs(_ptr(k, "cache.k", dev, bf16, shape), _ptr(cache.v, "cache.v", dev, bf16, shape), None, None, pages, page,
                           heads, d, KV_BF16)
    if cache.k_scales is None or cache.v_scales is None:
        raise ValueError("an MXFP8 cache has scales of its keys and of its values")
    u8, blocks = torch.uint8, (pages, heads, page, d // 32)
    return KvCacheArgs(_ptr(k, "cache.k", dev, u8, shape), _ptr(cache.v, "cache.v", dev, u8, shape),
                       _ptr(cache.k_scales, "cache.k_scales", dev, u8, blocks),
                       _ptr(cache.v_scales, "cache.v_scales", dev, u8, blocks), pages, page, heads, d, KV_MXFP8)


def page_plan(cached, added, block_table, free_pages, page_size, tokens, stream=None):
    """Pages, slots and positions of a step's new tokens -> PagePlan; ``block_table`` [requests, width] gets the new pages.

    cached, added: int32 [requests], tokens in the cache and new ones. free_pages: int32 [n], taken in the order of the
    requests; ``PagePlan.taken`` says how many were, and how many tokens are left without a page (their slots are -1).
    ``tokens`` is the length of slots and positions, at least the number of new tokens for all of them to be listed.
    """
    dev = _index(cached, "cached")
    i32, b = torch.int32, cached.shape[0] if cached.dim() == 1 else -1
    if b < 0:
        raise ValueError(f"cached must be [requests], got {tuple(cached.shape)}")
    pc, pa = _ptr(cached, "cached", dev, i32, (b,)), _ptr(added, "added", dev, i32, (b,))
    if block_table.dim() != 2 or block_table.shape[0] != b:
        raise ValueError(f"block_table must be [{b}, width], got {tuple(block_table.shape)}")
    width = block_table.shape[1]
    pt = _ptr(block_table, "block_table", dev, i32, (b, width))
    if free_pages.dim() != 1:
        raise ValueError(f"free_pages must be [n], got {tuple(free_pages.shape)}")
    n = free_pages.shape[0]
    pf = _ptr(free_pages, "free_pages", dev, i32, (n,))
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    handle, ctx = _on(dev, stream)
    with ctx:
        # one allocation: slots and positions from multiples of 16 bytes on
        pad = -tokens % 4
        buf = cached.new_empty(2 * (tokens + pad) + 2 * b + 3)
        slots, _, positions, _, starts, lengths, taken = buf.split_with_sizes((tokens, pad, tokens, pad, b + 1, b, 2))
        at = buf.data_ptr()
        pos = at + 4 * (tokens + pad)
        end = pos + 4 * (tokens + pad)
        st = _lib().mxq_page_plan(pc, pa, pt, pf, b, width, n, page_size, tokens, at, pos, end, end + 4 * (b + 1),
                                  end + 4 * (2 * b + 1), handle)
    _check(st, "page_plan")
    return PagePlan(slots, positions, starts, lengths, taken)


def rotary_qkv(qkv, heads, kv_heads, head_dim, positions=None, freqs=None, axis=None, interleaved=False,
               norm=ROTARY_NORM_NONE, q_weight=None, k_weight=None, eps=1e-6, q=None, k=None, write_k=True, cache=None,
               slots=None, stream=None):
    """RMS norm and rotary positions of stacked q/k/v rows -> (q [M, heads, D], k [M, kv_heads, D]), None for what is not there.

    qkv: bf16 [M, (heads + 2 kv_heads) D], rows may be strided. Pair p of a head turns by positions[axis[p], m] * freqs[p]
    (positions int32 [axes, M] or [M], freqs float64 [pairs], axis int32 [pairs], all on axis 0 if None); without freqs nothing turns.
    norm: none, over a row's heads (weights [heads D], [kv_heads D]) or per head (weights [D]). ``cache`` (KvCache) with
    ``slots`` int32 [M] takes k and v; ``write_k=False`` then leaves the dense k out. q and k may be given, also as views of
    qkv itself (its first heads * D and next kv_heads * D columns): in place.
    """
    dev = _index(qkv, "qkv")
    if qkv.dim() != 2:
        raise ValueError("qkv must be 2-D [rows, (heads + 2 kv_heads) * head_dim]")
    m, width = qkv.shape
    if heads < 0 or kv_heads < 0 or width != (heads + 2 * kv_heads) * head_dim:
        raise ValueError(f"qkv must have {(heads + 2 * kv_heads) * head_dim} columns, got {width}")
    px, ldx = _rows(qkv, "qkv", dev, (m, width))
    bf16 = torch.bfloat16
    pp = pf = pax = None
    axes = pairs = 0
    ld_pos = m
    if freqs is not None:
        if freqs.dim() != 1:
            raise ValueError("freqs must be [pairs]")
        pairs = freqs.shape[0]
        pf = _ptr(freqs, "freqs", dev, torch.float64, (pairs,))
        if positions is None or positions.dim() not in (1, 2):
            raise ValueError("a rotation needs positions [axes, M] or [M]")
        axes = positions.shape[0] if positions.dim() == 2 else 1
        pp = _ptr(positions, "positions", dev, torch.int32, (axes, m) if positions.dim() == 2 else (m,))
        pax = _ptr(axis, "axis", dev, torch.int32, (pairs,))
    elif positions is not None or axis is not None:
        raise ValueError("positions and axis belong to a rotation (freqs)")
    pqw = pkw = None
    if q_weight is not None:
        pqw = _ptr(q_weight, "q_weight", dev, bf16, (heads * head_dim if norm == ROTARY_NORM_ROW else head_dim,))
    if k_weight is not None:
        pkw = _ptr(k_weight, "k_weight", dev, bf16, (kv_heads * head_dim if norm == ROTARY_NORM_ROW else head_dim,))
    if (cache is None) != (slots is None):
        raise ValueError("cache and slots belong together")
    if cache is not None:
        c = _cache_args(cache, dev)
        ps = _ptr(slots, "slots", dev, torch.int32, (m,))
    else:
        c = ps = None
    if k is not None and not write_k:
        raise ValueError("k is an output of a call with write_k")
    handle, ctx = _on(dev, stream)
    with ctx:
        pq = pk = None
        ldq = ldk = 0
        if heads > 0:
            if q is None:
                q = qkv.new_empty((m, heads, head_dim))
                pq, ldq = q.data_ptr(), heads * head_dim
            else:
                pq, ldq = _heads(q, "q", dev, m, heads, head_dim)
        elif q is not None:
            raise ValueError("q is an output of a call with heads")
        if kv_heads > 0 and write_k:
            if k is None:
                k = qkv.new_empty((m, kv_heads, head_dim))
                pk, ldk = k.data_ptr(), kv_heads * head_dim
            else:
                pk, ldk = _heads(k, "k", dev, m, kv_heads, head_dim)
        elif k is not None:
            raise ValueError("k is an output of a call with kv_heads")
        args = RotaryArgs(px, pp, pf, pax, pqw, pkw, pq, pk, ps, m, ldx, ldq, ldk, ld_pos, heads, kv_heads, head_dim, axes, pairs,
                          int(interleaved), norm, eps)
        st = _lib().mxq_rotary_qkv(args, c, handle)
    _check(st, "rotary_qkv")
    return q, k


def _window(left, right, sinks):
    for n, v in (("window", left), ("window", right)):
        if v < -1:
            raise ValueError(f"{n} counts tokens, or -1 for no limit")
    if sinks < 0:
        raise ValueError("sinks must not be negative")
    return tuple(min(v, 1 << 62) for v in (left, right, sinks))


def attention(q, k, v, starts_q=None, starts_k=None, scale=None, window=(-1, -1), sinks=0, out=None, stream=None):
    """softmax(scale q k^T) v over what each query sees -> out bf16 [Mq, heads, D].

    q [Mq, heads, D], k and v [Mk, kv_heads, D], bf16, heads side by side, rows may be strided (views of a stacked projection).
    starts_q, starts_k: int32 [sequences + 1], the rows where sequences start and the last one ends; without them all rows are
    one sequence. A sequence's queries are the last of its positions; with ``window = (left, right)`` the one at p sees keys
    p - left .. p + right (-1: no limit, right 0: causal) and the first ``sinks`` ones up to p + right. Rows that see nothing
    are zeros; rows of ``out`` behind the last sequence stay, which in an output that the call allocates means that they hold
    anything. scale: 1 / sqrt(D) by default. ``out`` may not overlap an input.
    """
    dev = _index(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be 3-D [rows, heads, head_dim]")
    mq, heads, d = q.shape
    mk, kv_heads = k.shape[0], k.shape[1]
    pq, ldq = _heads(q, "q", dev)
    pk, ldk = _heads(k, "k", dev, mk, kv_heads, d)
    pv, ldv = _heads(v, "v", dev, mk, kv_heads, d)
    psq = psk = None
    sequences = 1
    if starts_q is not None or starts_k is not None:
        if starts_q is None or starts_k is None:
            raise ValueError("starts_q and starts_k belong together")
        if starts_q.dim() != 1 or starts_q.shape[0] < 1:
            raise ValueError(f"starts_q must be [sequences + 1], got {tuple(starts_q.shape)}")
        n = starts_q.shape[0]
        sequences = n - 1
        psq, psk = _ptr(starts_q, "starts_q", dev, torch.int32, (n,)), _ptr(starts_k, "starts_k", dev, torch.int32, (n,))
    left, right, sinks = _window(*window, sinks)
    handle, ctx = _on(dev, stream)
    with ctx:
        if out is None:
            out = q.new_empty((mq, heads, d))
            po, ldo = out.data_ptr(), heads * d
        else:
            po, ldo = _heads(out, "out", dev, mq, heads, d)
        args = AttentionArgs(pq, pk, pv, psq, psk, po, sequences, mq, mk, ldq, ldk, ldv, ldo, left, right, sinks, heads, kv_heads, d,
                             1.0 / math.sqrt(d) if scale is None else scale)
        need = ctypes.c_size_t()
        _check(_lib().mxq_attention_workspace_bytes(args, need), "attention")
        ws = torch.empty(need.value, dtype=torch.uint8, device=q.device) if need.value else None
        st = _lib().mxq_attention(args, ws.data_ptr() if need.value else None, need.value, handle)
    _check(st, "attention")
    return out


def attention_paged(q, cache, block_table, lengths, scale=None, window=-1, sinks=0, out=None, stream=None):
    """Attention of one new token per sequence over a paged cache -> out bf16 [sequences, heads, D].

    q [sequences, heads, D], at position lengths[b] - 1 of sequence b, whose keys and values are the first lengths[b] tokens of
    the pages block_table[b] (int32 [sequences, width]); the new token's own k and v are in the cache already (rotary_qkv).
    ``window`` is the number of earlier tokens that it sees (-1: all), besides the first ``sinks`` ones. ``out`` may not overlap an
    input.
    """
    dev = _index(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be 3-D [sequences, heads, head_dim]")
    b, heads, d = q.shape
    c = _cache_args(cache, dev)
    if c.head_dim != d:
        raise ValueError(f"q has heads of {d}, the cache of {c.head_dim}")
    pq, ldq = _heads(q, "q", dev)
    if block_table.dim() != 2 or block_table.shape[0] != b:
        raise ValueError(f"block_table must be [{b}, width], got {tuple(block_table.shape)}")
    width = block_table.shape[1]
    pt = _ptr(block_table, "block_table", dev, torch.int32, (b, width))
    pl = _ptr(lengths, "lengths", dev, torch.int32, (b,))
    left, _, sinks = _window(window, -1, sinks)
    handle, ctx = _on(dev, stream)
    with ctx:
        if out is None:
            out = q.new_empty((b, heads, d))
            po, ldo = out.data_ptr(), heads * d
        else:
            po, ldo = _heads(out, "out", dev, b, heads, d)
        args = PagedArgs(pq, pt, pl, po, b, width, ldq, ldo, left, sinks, heads, 1.0 / math.sqrt(d) if scale is None else scale)
        need = ctypes.c_size_t()
        _check(_lib().mxq_attention_paged_workspace_bytes(args, c, need), "attention_paged")
        ws = torch.empty(need.value, dtype=torch.uint8, device=q.device) if need.value else None
        st = _lib().mxq_attention_paged(args, c, ws.data_ptr() if need.value else None, need.value, handle)
    _check(st, "attention_paged")
    return out
