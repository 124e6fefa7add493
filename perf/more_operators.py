"""Measured cases of the attention half of a transformer block, between its stacked q/k/v projection and its output projection.

Four operators:

* ``plan``       page_plan: pages, slots and positions of a step's new tokens in a paged key-value cache, from the requests'
                 lengths;
* ``rotary``     rotary_qkv: RMS norm of q and k, rotary positions of one or several axes, k and v into the cache;
* ``attention``  attention: ragged sequences of tokens, grouped heads, sliding windows and sinks;
* ``paged``      attention_paged: one new token per sequence against a paged cache, bf16 or MXFP8.

``own`` chooses between the library's kernels and the plain form, which is elementary torch arithmetic in fp32 (angles in
64 bits). A cache is [pages, kv heads, page size, head size]; in MXFP8 it holds E4M3 codes with one power-of-two scale per
32 elements of a head, and comes back here as the bf16 values that it stands for (all of them are bf16 numbers).
"""

import math
import random

import torch

own = False  # the library's operators (True) or the plain form (False)

EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one step of 64 sequences that decode together: a slot for each sequence's new token; latency counts
        {"name": "plan decode 64", "op": "plan", "requests": 64, "cached": 131072, "new": 64, "tokens": 64, "page": 16,
         "free": 64, "width": 1024, "ragged": 1},
        # a scheduler's largest step: prompts of a thousand requests, some of them with a cached beginning
        {"name": "plan prefill 1000", "op": "plan", "requests": 1000, "cached": 300007, "new": 200003, "tokens": 204800,
         "page": 64, "free": 8192, "width": 128, "ragged": 2},
        # one token of a decoder with grouped heads: norm per head, one axis, into its cache slot; latency counts
        {"name": "rotary token", "op": "rotary", "m": 1, "heads": 40, "kv_heads": 8, "d": 128, "style": "half", "axes": 1,
         "pairs": 64, "norm": "head", "cache": "bf16", "page": 16, "dense_k": False, "padded": 0},
        # a 720p video transformer's self-attention: norm over the row, time x height x width; the largest stream
        {"name": "rotary 720p video", "op": "rotary", "m": 75600, "heads": 40, "kv_heads": 40, "d": 128, "style": "interleaved",
         "axes": 3, "pairs": 64, "norm": "row", "cache": "none", "page": 16, "dense_k": True, "padded": 0},
        # prompts of several requests, an odd number of tokens, a padded end: into the cache and onwards to attention
        {"name": "rotary prompts", "op": "rotary", "m": 8195, "heads": 40, "kv_heads": 8, "d": 128, "style": "half", "axes": 1,
         "pairs": 64, "norm": "head", "cache": "bf16", "page": 64, "dense_k": True, "padded": 13},
        # 480p video self-attention: every token sees every token; the largest product
        {"name": "attention 480p video", "op": "attention", "sequences": 1, "mq": 32760, "mk": 32760, "heads": 40, "kv_heads": 40,
         "d": 128, "left": -1, "right": -1, "sinks": 0, "ragged": 0},
        # 480p video tokens of two requests against their texts
        {"name": "attention text", "op": "attention", "sequences": 2, "mq": 65520, "mk": 741, "heads": 40, "kv_heads": 40, "d": 128,
         "left": -1, "right": -1, "sinks": 0, "ragged": 3},
        # prompts together, causal, a sliding window and the first tokens of each
        {"name": "attention prompts window", "op": "attention", "sequences": 5, "mq": 16387, "mk": 16387, "heads": 40,
         "kv_heads": 8, "d": 128, "left": 1023, "right": 0, "sinks": 4, "ragged": 4},
        # a few new tokens at the end of a long context, heads of 64: few rows, a long axis
        {"name": "attention few rows", "op": "attention", "sequences": 1, "mq": 37, "mk": 30011, "heads": 64, "kv_heads": 8,
         "d": 64, "left": -1, "right": 0, "sinks": 0, "ragged": 0},
        # one sequence, a long cache
        {"name": "paged long", "op": "paged", "sequences": 1, "cached": 131071, "heads": 40, "kv_heads": 8, "d": 128,
         "cache": "bf16", "page": 16, "left": -1, "sinks": 0, "ragged": 5},
        # a serving step of 64 sequences of very different lengths, MXFP8 cache
        {"name": "paged batch mxfp8", "op": "paged", "sequences": 64, "cached": 262147, "heads": 40, "kv_heads": 8, "d": 128,
         "cache": "mxfp8", "page": 64, "left": -1, "sinks": 0, "ragged": 6},
        # a sliding window with sinks over longer caches, heads of 64; latency counts
        {"name": "paged window", "op": "paged", "sequences": 9, "cached": 60013, "heads": 64, "kv_heads": 8, "d": 64,
         "cache": "bf16", "page": 32, "left": 2047, "sinks": 4, "ragged": 7},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, ragged = rng.choice(["plan", "rotary", "attention", "paged"]), rng.randint(0, 1 << 30)
    heads, kv_heads, d = rng.choice([(40, 40, 128), (40, 8, 128), (64, 64, 64), (64, 8, 64), (10, 2, 128), (5, 5, 128), (16, 1, 64),
                                     (12, 4, 128)])
    if op == "plan":
        requests, page = _spread(rng, 1, 2000), rng.choice([16, 32, 64, 128])
        new, cached = _spread(rng, requests, 100000 + requests), _spread(rng, 1, 500000)
        need = new // page + requests
        return {"op": op, "requests": requests, "cached": cached, "new": new, "tokens": new + _spread(rng, 1, 2000), "page": page,
                "free": need if rng.random() < 0.8 else max(1, need // 2), "width": _spread(rng, 64, 2048), "ragged": ragged}
    if op == "rotary":
        m, cache = _spread(rng, 1, 20000), rng.choice(["none", "bf16", "mxfp8"])
        style, axes = rng.choice([("half", 1), ("half", 3), ("interleaved", 1), ("interleaved", 3)])
        return {"op": op, "m": m, "heads": heads, "kv_heads": kv_heads, "d": d, "style": style, "axes": axes,
                "pairs": rng.choice([d // 2, d // 2, d // 4]), "norm": rng.choice(["none", "row", "head"]), "cache": cache,
                "page": rng.choice([16, 32, 64, 128]), "dense_k": cache == "none" or rng.random() < 0.5,
                "padded": rng.randint(0, min(7, m - 1))}
    if op == "attention":
        sequences = _spread(rng, 1, 30)
        mq = _spread(rng, sequences, 9000 + sequences)
        same = rng.random() < 0.5
        left, right, sinks = rng.choice([(-1, -1, 0), (-1, 0, 0), (_spread(rng, 16, 4000), 0, rng.choice([0, 1, 4, 70])),
                                         (_spread(rng, 16, 1000), _spread(rng, 16, 1000), rng.choice([0, 4]))])
        return {"op": op, "sequences": sequences, "mq": mq, "mk": mq if same else _spread(rng, 1, 12000), "heads": heads,
                "kv_heads": kv_heads, "d": d, "left": left, "right": right, "sinks": sinks, "ragged": ragged}
    sequences = _spread(rng, 1, 200)
    left, sinks = rng.choice([(-1, 0), (-1, 0), (_spread(rng, 16, 8000), rng.choice([0, 1, 4, 70]))])
    return {"op": op, "sequences": sequences, "cached": _spread(rng, 8 * sequences, 100000 + 8 * sequences), "heads": heads,
            "kv_heads": kv_heads, "d": d, "cache": rng.choice(["bf16", "mxfp8"]), "page": rng.choice([16, 32, 64, 128]),
            "left": left, "sinks": sinks, "ragged": ragged}


def _parts(total, count, seed, least=0):
    """`count` whole numbers of at least `least` that sum to `total`, a few of them much larger than the others; the same for
    the same seed."""
    rng = random.Random(seed)
    weights = [math.exp(rng.gauss(0.0, 1.0)) for _ in range(count)]
    spare, whole = total - least * count, sum(weights)
    ends, acc = [0], 0.0
    for w in weights:
        acc += w
        ends.append(int(round(spare * acc / whole)))
    ends[-1] = spare
    return [least + b - a for a, b in zip(ends, ends[1:])]


def _plan_lengths(case):
    return _parts(case["cached"], case["requests"], case["ragged"]), _parts(case["new"], case["requests"], case["ragged"] + 1, 1)


def _sequence_lengths(case):
    """Query and key counts of an attention case's sequences."""
    q = _parts(case["mq"], case["sequences"], case["ragged"])
    return q, q if case["mq"] == case["mk"] else _parts(case["mk"], case["sequences"], case["ragged"] + 1)


def _cached_lengths(case):
    return _parts(case["cached"], case["sequences"], case["ragged"], 1)


def _visible_pairs(nq, nk, left, right, sinks):
    """Visible (query, key) pairs of a sequence."""
    if nq == 0 or nk == 0:
        return 0
    p = torch.arange(nq, dtype=torch.float64) + (nk - nq)
    last = (p + right).clamp(max=nk - 1) if right >= 0 else torch.full_like(p, nk - 1)
    first = (p - left).clamp(min=0) if left >= 0 else torch.zeros_like(p)
    window = (last - first + 1).clamp(min=0)
    return int((window + (torch.minimum(last + 1, torch.minimum(first, torch.full_like(p, min(sinks, nk))))).clamp(min=0)).sum())


def work(case):
    op = case["op"]
    if op == "plan":
        b, taken = case["requests"], case["new"] // case["page"]
        return {"bytes": 16 * b + 8 * case["tokens"] + 8 * taken, "flops": 4 * case["tokens"]}
    h, g, d = case["heads"], case["kv_heads"], case["d"]
    if op == "rotary":
        m, cached = case["m"], case["m"] - case["padded"]
        moved = m * (h + g) * d * 2 + m * h * d * 2 + (m * g * d * 2 if case["dense_k"] else 0) + 4 * m * max(1, case["axes"])
        if case["cache"] != "none":
            moved += cached * g * d * 2 + 2 * cached * g * (2 * d if case["cache"] == "bf16" else d + d // 32) + 4 * m
        return {"bytes": moved, "flops": 10 * m * (h + g) * d}
    if op == "attention":
        pairs = sum(_visible_pairs(a, b, case["left"], case["right"], case["sinks"]) for a, b in zip(*_sequence_lengths(case)))
        return {"bytes": 4 * case["mq"] * h * d + 4 * case["mk"] * g * d, "flops": 4 * d * h * pairs}
    keys = sum(_visible_pairs(1, n, case["left"], -1, case["sinks"]) for n in _cached_lengths(case))
    row = 2 * d if case["cache"] == "bf16" else d + d // 32
    return {"bytes": 2 * keys * g * row + 4 * case["sequences"] * h * d, "flops": 4 * d * h * keys}


# ----------------------------------------------------------------- inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lengths):
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    return _ints(ends)


def _page_counts(lengths, page):
    return [-(-n // page) for n in lengths]


def _tables(g, counts, width, spare):
    """(block table [requests, width] of distinct pages in any order, -1 behind each request's, `spare` further pages)."""
    total = sum(counts)
    pages = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    n = _ints(counts)
    ends = torch.cumsum(n, 0)
    j = torch.arange(width, device="cuda")[None]
    at = (ends - n)[:, None] + j
    table = torch.where(j < n[:, None], pages[at.clamp(max=total + spare - 1)], torch.full_like(at, -1).int())
    return table.to(torch.int32).contiguous(), pages[total:].contiguous()


def _exponents(v):
    """Exponent of the MX scale of each 32 of v's last axis, E4M3 elements (largest exponent 8)."""
    amax = v.float().unflatten(-1, (-1, 32)).abs().amax(dim=-1)
    return torch.where(amax > 0, torch.frexp(amax).exponent - 9, torch.full_like(amax, -127, dtype=torch.int32)).clamp(min=-127)


def _mxfp8(v):
    """bf16 [..., D] -> (E4M3 codes uint8 [..., D], E8M0 scales uint8 [..., D / 32])."""
    e = _exponents(v)
    q = torch.ldexp(v.float().unflatten(-1, (-1, 32)), -e[..., None]).clamp(-448.0, 448.0)
    return q.flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _of_mxfp8(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return torch.ldexp(v, scales.int()[..., None] - 127).flatten(-2).to(torch.bfloat16)


def _keys(g, *shape):
    """Normal keys with one channel in 64 four times as large."""
    k = _randn(g, *shape)
    k[..., torch.randperm(shape[-1], generator=g, device="cuda")[: shape[-1] // 64]] *= 4.0
    return k.to(torch.bfloat16)


def _inputs(case, seed):
    g, op, t = _gen(seed), case["op"], {}
    if op == "plan":
        cached, new = _plan_lengths(case)
        t["cached"], t["new"] = _ints(cached), _ints(new)
        t["table"], t["free"] = _tables(g, [min(n, case["width"]) for n in _page_counts(cached, case["page"])], case["width"],
                                        case["free"])
        return t
    h, kv, d = case["heads"], case["kv_heads"], case["d"]
    if op == "rotary":
        m, pairs, axes = case["m"], case["pairs"], case["axes"]
        x = _randn(g, m, (h + 2 * kv) * d)
        x[:, torch.randperm(x.shape[1], generator=g, device="cuda")[: max(1, x.shape[1] // 200)]] *= 10.0
        t["qkv"] = x.to(torch.bfloat16)
        per_axis = [pairs - (axes - 1) * (pairs // 3), pairs // 3, pairs // 3][:axes]
        t["freqs"] = torch.tensor([THETA ** (-i / n) for n in per_axis for i in range(n)], dtype=torch.float64, device="cuda")
        t["axis"] = _ints([a for a, n in enumerate(per_axis) for _ in range(n)])
        tokens = torch.arange(m, device="cuda")
        if axes == 1:  # one axis: a context that may be a million tokens long
            t["positions"] = (tokens + torch.randint(0, 1000000, (1,), generator=g, device="cuda"))[None].to(torch.int32)
        else:  # time, height and width of a grid of 45 x 80 per frame
            t["positions"] = torch.stack([tokens // 3600, tokens // 80 % 45, tokens % 80]).to(torch.int32)
        wide = case["norm"] == "row"
        for name, heads in (("q_weight", h), ("k_weight", kv)):
            t[name] = None if case["norm"] == "none" else (1.0 + 0.1 * _randn(g, heads * d if wide else d)).to(torch.bfloat16)
        if case["cache"] != "none":
            pages = -(-m // case["page"]) + 3
            slots = torch.randperm(pages * case["page"], generator=g, device="cuda")[:m].to(torch.int32)
            slots[m - case["padded"]:] = -1
            t["slots"] = slots
            t["cache"] = tuple(_randn(g, pages, kv, case["page"], d).to(torch.bfloat16) for _ in range(2))
        return t
    if op == "attention":
        t["q"] = (1.5 * _randn(g, case["mq"], h, d)).to(torch.bfloat16)
        t["k"], t["v"] = _keys(g, case["mk"], kv, d), _randn(g, case["mk"], kv, d).to(torch.bfloat16)
        nq, nk = _sequence_lengths(case)
        t["starts_q"], t["starts_k"] = _starts(nq), _starts(nk)
        return t
    lengths = _cached_lengths(case)
    counts = _page_counts(lengths, case["page"])
    t["q"] = (1.5 * _randn(g, case["sequences"], h, d)).to(torch.bfloat16)
    t["table"], _ = _tables(g, counts, max(counts) + 3, 5)
    t["lengths"] = _ints(lengths)
    shape = (sum(counts) + 5, kv, case["page"], d)
    t["cache"] = _keys(g, *shape), _randn(g, *shape).to(torch.bfloat16)
    return t


def prepare(case, seed):
    """The tensors of a case; a quantized cache holds codes and scales, as the steps before left it."""
    s = _inputs(case, seed)
    s["case"] = case
    if case.get("cache") == "mxfp8":
        (kc, ks), (vc, vs) = (_mxfp8(c) for c in s["cache"])
        s["cache"] = kc, vc, ks, vs
    return s


# ------------------------------------------------------------------- runs ----

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _cache_values(cache):
    """A cache's keys and values in bf16."""
    return (_of_mxfp8(cache[0], cache[2]), _of_mxfp8(cache[1], cache[3])) if len(cache) == 4 else tuple(cache)


def _run_own(s):
    import mx_bit_quantized_amd as mxq

    case, op = s["case"], s["case"]["op"]
    if op == "plan":
        return (*mxq.page_plan(s["cached"], s["new"], s["table"], s["free"], case["page"], case["tokens"]), s["table"])
    if op == "rotary":
        norm = {"none": mxq.ROTARY_NORM_NONE, "row": mxq.ROTARY_NORM_ROW, "head": mxq.ROTARY_NORM_HEAD}[case["norm"]]
        kept = case["cache"] != "none"
        q, k = mxq.rotary_qkv(s["qkv"], case["heads"], case["kv_heads"], case["d"], s["positions"], s["freqs"], s["axis"],
                              interleaved=case["style"] == "interleaved", norm=norm, q_weight=s["q_weight"],
                              k_weight=s["k_weight"], eps=EPS, write_k=case["dense_k"],
                              cache=mxq.KvCache(*s["cache"]) if kept else None, slots=s["slots"] if kept else None)
        return (q, k) + (_cache_values(s["cache"]) if kept else ())
    if op == "attention":
        return mxq.attention(s["q"], s["k"], s["v"], s["starts_q"], s["starts_k"], window=(case["left"], case["right"]),
                             sinks=case["sinks"])
    return mxq.attention_paged(s["q"], mxq.KvCache(*s["cache"]), s["table"], s["lengths"], window=case["left"],
                               sinks=case["sinks"])


# ------------------------------------------------------------- plain form ----

def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "plan":
        return _plain_plan(s, case)
    if op == "rotary":
        return _plain_rotary(s, case)
    if op == "attention":
        return _plain_attention(s, case)
    return _plain_paged(s, case)


def _plain_plan(s, case):
    page, width, table, free = case["page"], case["width"], s["table"], s["free"].long()
    c, n = s["cached"].long(), s["new"].long()
    have, want = ((v + page - 1).div(page, rounding_mode="floor").clamp(max=width) for v in (c, c + n))
    need = want - have
    base = torch.cumsum(need, 0) - need
    j = torch.arange(width, device=c.device)[None]
    at = base[:, None] + j - have[:, None]
    fresh = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], torch.full_like(at, -1))
    table = torch.where((j >= have[:, None]) & (j < want[:, None]), fresh, table.long()).to(torch.int32)
    starts = torch.cat([torch.zeros_like(n[:1]), torch.cumsum(n, 0)])
    t = torch.arange(case["tokens"], device=c.device)
    b = (torch.searchsorted(starts, t, right=True) - 1).clamp(max=case["requests"] - 1)
    live = t < starts[-1]
    position = torch.where(live, c[b] + t - starts[b], torch.zeros_like(t))
    column = position.div(page, rounding_mode="floor")
    held = table[b, column.clamp(max=width - 1)].long()
    slots = torch.where(live & (column < width) & (held >= 0), held * page + position % page, torch.full_like(t, -1))
    taken = torch.stack([need.sum().clamp(max=free.numel()), (live & (slots < 0)).sum()])
    return (*(v.to(torch.int32) for v in (slots, position, starts, c + n, taken)), table)


def _plain_turned(x, norm, weight, cos, sin, style):
    """Norm and rotation of fp32 [m, heads, d]."""
    m, heads, d = x.shape
    if norm == "row":
        x = x.reshape(m, heads * d)
    if norm != "none":
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()
    x = x.view(m, heads, d)
    pairs = cos.shape[-1]
    turned, rest = x[..., : 2 * pairs], x[..., 2 * pairs:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if style == "interleaved" else (turned[..., :pairs], turned[..., pairs:])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], dim=-1).flatten(-2) if style == "interleaved" else torch.cat([a, b], dim=-1)
    return torch.cat([turned, rest], dim=-1).to(torch.bfloat16)


def _plain_rotary(s, case):
    m, h, kv, d, page = case["m"], case["heads"], case["kv_heads"], case["d"], case["page"]
    angle = (s["positions"].double()[s["axis"].long()] * s["freqs"][:, None]).t()[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    x = s["qkv"].view(m, h + 2 * kv, d)
    q = _plain_turned(x[:, :h].float(), case["norm"], s["q_weight"], cos, sin, case["style"])
    k = _plain_turned(x[:, h:h + kv].float(), case["norm"], s["k_weight"], cos, sin, case["style"])
    dense = k if case["dense_k"] else None
    if case["cache"] == "none":
        return q, dense
    v = x[:, h + kv:]
    kept = s["slots"] >= 0
    at = s["slots"][kept].long()
    new = (k[kept], v[kept])
    if case["cache"] == "mxfp8":
        (kc, ks), (vc, vs) = _mxfp8(new[0]), _mxfp8(new[1])
        new = (kc, vc, ks, vs)
    for held, rows in zip(s["cache"], new):
        held[at // page, :, at % page] = rows
    return (q, dense) + _cache_values(s["cache"])


def _plain_visible(p, j, nk, left, right, sinks):
    """Which keys j < nk a query at position p sees."""
    seen = j < nk
    if right >= 0:
        seen = seen & (j <= p + right)
    if left >= 0:
        seen = seen & ((j >= p - left) | (j < sinks))
    return seen


def _plain_softmax_product(score, seen, v):
    """softmax(score) v over the visible keys, zeros where there are none."""
    if seen is not None:
        score.masked_fill_(~seen, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    weight = score.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = weight.sum(dim=-1, keepdim=True)
    return (weight @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_attention(s, case):
    (mq, h, d), kv, mk = s["q"].shape, case["kv_heads"], case["mk"]
    if mk == 0:
        return torch.zeros_like(s["q"])
    group = h // kv
    seen = None
    if case["sequences"] > 1 or case["left"] >= 0 or case["right"] >= 0:
        sq, sk = s["starts_q"].long(), s["starts_k"].long()
        i, j = torch.arange(mq, device=sq.device), torch.arange(mk, device=sq.device)
        bi, bj = torch.searchsorted(sq, i, right=True) - 1, torch.searchsorted(sk, j, right=True) - 1
        nq, nk = sq.diff(), sk.diff()
        seen = _plain_visible((i - sq[bi] + nk[bi] - nq[bi])[:, None], (j - sk[bj])[None], nk[bj][None], case["left"],
                              case["right"], case["sinks"]) & (bi[:, None] == bj[None])
    out = torch.empty_like(s["q"])
    step = max(1, (1 << 32) // (mq * mk * group))  # kv heads at a time: the scores of all of them would not fit
    for g in range(0, kv, step):
        q = s["q"][:, g * group:(g + step) * group].float().unflatten(1, (-1, group)).permute(1, 2, 0, 3).contiguous()
        k, v = (s[n][:, g:g + step].float().permute(1, 0, 2)[:, None].contiguous() for n in ("k", "v"))
        score = (q.flatten(1, 2)[:, None] @ k.mT.contiguous()).unflatten(2, (group, mq))[:, 0]
        o = _plain_softmax_product(score.mul_(d ** -0.5), seen, v)
        out[:, g * group:(g + step) * group] = o.permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16)
    return out


def _plain_paged(s, case):
    (b, h, d), kv = s["q"].shape, case["kv_heads"]
    at = s["table"].long().clamp(min=0)
    if case["cache"] == "mxfp8":
        held = [_of_mxfp8(c[at], e[at]) for c, e in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3]))]
    else:
        held = [c[at] for c in s["cache"]]
    k, v = (c.float().transpose(1, 2).flatten(2, 3) for c in held)  # [b, kv, keys, d]
    n = s["lengths"].long()[:, None]
    seen = _plain_visible(n - 1, torch.arange(k.shape[2], device=n.device)[None], n, case["left"], -1, case["sinks"])
    q = s["q"].float().unflatten(1, (kv, -1))
    o = _plain_softmax_product((q @ k.mT.contiguous()) * d ** -0.5, seen[:, None, None], v)
    return o.flatten(1, 2).to(torch.bfloat16)


# ---------------------------------------------------- definition in 64 bits ----

def _exact_heads(x, weight, case, angle):
    """float64 [m, heads, d] normed and turned: pairs as complex numbers times exp(i angle)."""
    if case["norm"] != "none":
        dims = (1, 2) if case["norm"] == "row" else (2,)
        x = x / torch.sqrt(x.square().mean(dims, keepdim=True) + EPS) * weight.double().view(-1, x.shape[2])
    pairs = angle.shape[1]
    first = torch.arange(pairs, device=x.device) * (2 if case["style"] == "interleaved" else 1)
    second = first + (1 if case["style"] == "interleaved" else pairs)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_mxfp8(v):
    """The values that MXFP8 gives to float64 [..., D] holding bf16 values."""
    b = v.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(top)).clamp(-119, 135) - 8)
    r = b / scale
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.clamp(torch.round(r / step) * step, -448.0, 448.0) * scale).flatten(-2)


def _exact_softmax(score, v):
    """Rows of probabilities times v, from scores of -inf where a key is not visible."""
    return torch.nan_to_num(torch.exp(score - torch.logsumexp(score, -1, keepdim=True)), nan=0.0) @ v


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    t = _inputs(case, seed)
    h, kv, d, group = case["heads"], case["kv_heads"], case["d"], case["heads"] // case["kv_heads"]
    if case["op"] == "rotary":
        m = case["m"]
        x = t["qkv"].double().view(m, h + 2 * kv, d)
        angle = torch.stack([t["positions"][a].double() * f for a, f in zip(t["axis"].tolist(), t["freqs"].tolist())], 1)
        q, k = _exact_heads(x[:, :h], t["q_weight"], case, angle), _exact_heads(x[:, h:h + kv], t["k_weight"], case, angle)
        dense = k if case["dense_k"] else None
        if case["cache"] == "none":
            return q, dense
        held = [c.double() for c in t["cache"]]
        new = [k, x[:, h + kv:]]
        if case["cache"] == "mxfp8":
            held = [_exact_mxfp8(c) for c in held]
            new = [_exact_mxfp8(k.to(torch.bfloat16).double()), _exact_mxfp8(new[1])]
        for row in range(2):
            flat = held[row].transpose(1, 2).reshape(-1, kv, d).clone()
            kept = t["slots"] >= 0
            flat[t["slots"][kept].long()] = new[row][kept]
            held[row] = flat.view(-1, case["page"], kv, d).transpose(1, 2)
        return q, dense, held[0], held[1]
    left, right, sinks = case["left"], case.get("right", -1), case["sinks"]

    def attend(q, k, v, p):
        """Heads' queries [n, d] at positions p against their keys [keys, d], all of one sequence, a few rows at a time."""
        rows, out = max(1, (1 << 28) // max(1, k.shape[0])), torch.zeros_like(q)
        j = torch.arange(k.shape[0], device=q.device)
        for r in range(0, q.shape[0], rows):
            at = p[r:r + rows, None]
            low = at - left if left >= 0 else at * 0
            high = at + right if right >= 0 else at * 0 + k.shape[0]
            hidden = (j > high) | ((j < low) & (j >= sinks))
            out[r:r + rows] = _exact_softmax((q[r:r + rows] @ k.t() / math.sqrt(d)).masked_fill(hidden, -math.inf), v)
        return out

    out = torch.zeros(t["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "attention":
        nq, nk = _sequence_lengths(case)
        bounds = [(sum(nq[:b]), nq[b], sum(nk[:b]), nk[b]) for b in range(case["sequences"])]
    else:
        bounds = [(b, 1, None, n) for b, n in enumerate(_cached_lengths(case))]
        held = [_exact_mxfp8(c.double()).to(torch.bfloat16) if case["cache"] == "mxfp8" else c for c in t["cache"]]
    for b, (q0, qn, k0, kn) in enumerate(bounds):
        if qn == 0 or kn == 0:
            continue
        p = (torch.arange(qn, device="cuda") + kn - qn).repeat(group)
        if case["op"] == "attention":
            k, v = t["k"][k0:k0 + kn], t["v"][k0:k0 + kn]
        else:
            pages = t["table"][b, : -(-kn // case["page"])].long()
            k, v = (c[pages].transpose(1, 2).reshape(-1, kv, d)[:kn] for c in held)
        for g in range(kv):
            q = t["q"][q0:q0 + qn, g * group:(g + 1) * group].double().transpose(0, 1).reshape(-1, d)
            o = attend(q, k[:, g].double(), v[:, g].double(), p)
            out[q0:q0 + qn, g * group:(g + 1) * group] = o.view(group, qn, d).transpose(0, 1)
    return out
