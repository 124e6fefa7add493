"""The attention half of a block: page plan, norm and rotary positions, MXFP8 blocks, windowed attention.

Each function is its operator's definition, element by element or row by row in float64 (whole numbers for
the plan), of numpy arrays. ``attention_rows`` also returns, per output element, the weighted mean of |v|
that tolerances are stated in.
"""

import numpy as np

from .formats import e4m3fn_decode, e4m3fn_encode, round_to_binary_format

HIDDEN = -np.inf


def page_plan(cached, added, table, free, page, tokens):
    """(slots, positions, starts, lengths, taken, table after): request by request, token by token."""
    table = np.array(table, np.int64)
    width = table.shape[1]
    free, used = list(free), 0
    slots, positions, starts, lengths, unplaced = [], [], [0], [], 0
    for r, (c, n) in enumerate(zip(cached, added)):
        c, n = max(int(c), 0), max(int(n), 0)
        have, want = (min(-(-x // page), width) for x in (c, c + n))
        for col in range(have, want):
            table[r, col] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + n):
            held = table[r, p // page] if p // page < width else -1
            unplaced += held < 0
            slots.append(held * page + p % page if held >= 0 else -1)
            positions.append(p)
        starts.append(starts[-1] + n)
        lengths.append(c + n)
    spare = max(0, tokens - len(slots))
    slots, positions = (slots + [-1] * spare)[:tokens], (positions + [0] * spare)[:tokens]
    return slots, positions, starts, lengths, [min(used, len(free)), unplaced], table


def rms_norm(x, weight, eps):
    """x / sqrt(mean x^2 + eps) * weight over the last axis."""
    n = x / np.sqrt(np.mean(np.square(x), axis=-1, keepdims=True) + eps)
    return n if weight is None else n * weight


def rotate(x, angle, interleaved):
    """Heads [..., D] with pair p turned by angle[..., p]; elements behind the pairs stay."""
    pairs = angle.shape[-1]
    out = np.array(x, np.float64)
    first, second = (np.s_[0:2 * pairs:2], np.s_[1:2 * pairs:2]) if interleaved else (np.s_[:pairs], np.s_[pairs:2 * pairs])
    a, b = x[..., first], x[..., second]
    out[..., first] = a * np.cos(angle) - b * np.sin(angle)
    out[..., second] = a * np.sin(angle) + b * np.cos(angle)
    return out


def mxfp8_quantize(x):
    """float64 [..., D] of bf16 values -> (E4M3 codes [..., D], E8M0 scales [..., D / 32]), uint8."""
    b = x.reshape(x.shape[:-1] + (-1, 32))
    amax = np.abs(b).max(axis=-1)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.floor(np.log2(amax)) - 8, -127.0).clip(-127, 127)
    q = round_to_binary_format(np.ldexp(b, -e.astype(int)[..., None]), 3, -6, 448.0)
    return e4m3fn_encode(q).reshape(x.shape), (e + 127).astype(np.uint8)


def mxfp8_dequantize(codes, scales):
    v = e4m3fn_decode(codes).reshape(codes.shape[:-1] + (-1, 32))
    return np.ldexp(v, scales.astype(int)[..., None] - 127).reshape(codes.shape)


def visible(p, keys, left, right, sinks):
    """Which of `keys` key positions a query at position p sees."""
    j = np.arange(keys)
    seen = np.ones(keys, bool) if right < 0 else j <= p + right
    return seen if left < 0 else seen & ((j >= p - left) | (j < sinks))


def attention_rows(q, k, v, first, left, right, sinks, scale):
    """One head: queries [n, D] at positions first .. against keys and values [m, D] -> (out, sum w |v|, largest sum |q k|).

    Hidden keys and values are not touched, whatever they hold.
    """
    out, mean, top = np.zeros(q.shape), np.zeros(q.shape), np.zeros(len(q))
    for i in range(len(q)):
        seen = visible(first + i, len(k), left, right, sinks)
        if not seen.any():
            continue
        ks, vs = k[seen], v[seen]
        s = scale * (ks @ q[i])
        w = np.exp(s - s.max())
        w /= w.sum()
        out[i], mean[i] = w @ vs, w @ np.abs(vs)
        top[i] = scale * (np.abs(ks) @ np.abs(q[i])).max()
    return out, mean, top
