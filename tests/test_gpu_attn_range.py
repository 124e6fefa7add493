"""GPU tests of the attention half at the ends of what its inputs may hold: very large and very small numbers, and where the
arithmetic leaves fp32's range. Tolerances: those of test_gpu_attn.py."""

import numpy as np
import pytest
import torch

import mx_bit_quantized_amd as mxq
import oracle
from test_gpu_attn import BF16, DEV, attention_check, gen, host, ints, randn, rotary_want, rotary_within, say, within
from test_gpu_check_finite import guard

pytestmark = pytest.mark.gpu


def reported(call):
    with guard(True), pytest.raises(mxq.MxqError) as e:
        call()
    assert e.value.status == mxq.ERR_NONFINITE


# ------------------------------------------------------- norms of rotary_qkv ----

NORMED = [(3, 4, 2, 64), (4, 128, 128, 128), (3, 170, 170, 128), (2051, 40, 8, 128)]  # one, two, four units a thread; two rows a step


def normed_case(m, heads, kv, d, norm, value):
    g = gen(heads + m)
    x = randn(g, m, (heads + 2 * kv) * d, scale=2.0)
    of = (heads * d, kv * d) if norm == 1 else (d, d)
    weights = [(1 + 0.2 * torch.randn(n, generator=g)).to(BF16) for n in of]
    if value is not None:
        x[1, 3 * d + 9] = value                    # q, head 3
        x[m - 1, (heads + kv - 1) * d + 40] = -value  # k, its last head
    call = lambda **more: mxq.rotary_qkv(x.to(DEV), heads, kv, d, norm=norm, q_weight=weights[0].to(DEV), k_weight=weights[1].to(DEV),
                                         **more)
    return x, weights, call


@pytest.mark.parametrize("norm", [mxq.ROTARY_NORM_ROW, mxq.ROTARY_NORM_HEAD])
@pytest.mark.parametrize("m, heads, kv, d", NORMED)
def test_rotary_norms_past_the_range(m, heads, kv, d, norm):
    """The row (or head) is NaN, dense and in the cache, everything else stays; the guard reports it."""
    say("norm range", m, heads, kv, d, norm)
    held = mxq.kv_cache(m // 16 + 1, kv, 16, d)
    want_q, want_k = normed_case(m, heads, kv, d, norm, None)[2]()
    call = normed_case(m, heads, kv, d, norm, 2e19)[2]
    q, k = call(cache=held, slots=ints(list(range(m))))
    bad_q, bad_k = torch.zeros(m, heads, dtype=torch.bool, device=DEV), torch.zeros(m, kv, dtype=torch.bool, device=DEV)
    bad_q[1, slice(None) if norm == mxq.ROTARY_NORM_ROW else 3] = True
    bad_k[m - 1, slice(None) if norm == mxq.ROTARY_NORM_ROW else kv - 1] = True
    kept = held.k.transpose(1, 2).reshape(-1, kv, d)[:m]
    for got, bad, want in ((q, bad_q, want_q), (k, bad_k, want_k), (kept, bad_k, want_k)):
        assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])
    reported(call)


@pytest.mark.parametrize("norm", [mxq.ROTARY_NORM_ROW, mxq.ROTARY_NORM_HEAD])
@pytest.mark.parametrize("m, heads, kv, d", NORMED)
def test_rotary_norms_inside_the_range(m, heads, kv, d, norm):
    """2^63, whose square is 2^126, among ordinary numbers."""
    say("norm inside", m, heads, kv, d, norm)
    x, weights, call = normed_case(m, heads, kv, d, norm, 2.0 ** 63)
    some = sorted({0, 1, m - 1})
    want = rotary_want(x[some], heads, kv, d, torch.zeros(0, dtype=torch.float64), [], None, weights, norm, False)
    q, k = call()
    rotary_within(q[some], want[0], "q")
    rotary_within(k[some], want[1], "k")


# -------------------------------------------------------- scales of attention ----

@pytest.mark.parametrize("d, group", [(64, 1), (128, 4)])
@pytest.mark.parametrize("scale", [1e-38, 1e-39, 1e-45, 1e-30])
def test_attention_scales_near_zero(scale, d, group):
    """Rows that see nothing of a part's first tile, other rows of their wave do, and a scale whose inverse overflows."""
    nq, nk, left = 40, 20000, 2946
    say("scale", scale, d, group)
    g = gen(d)
    q, k = randn(g, nq, group, d), randn(g, nk, 1, d)
    v = torch.zeros(nk, 1, d, dtype=BF16)
    v[17024:17088] = 8.0  # (in the first part of the keys; the rows' windows begin at 17014 to 17053)
    out = mxq.attention(q.to(DEV), k.to(DEV), v.to(DEV), window=(left, 0), scale=scale)
    attention_check(out, q, k, v, [(nq, nk)], left, 0, 0, scale, "scale")
    # ragged sequences of few keys, in one part
    lens = [(50, 200), (3, 1), (70, 70)]
    q, k, v = (randn(g, 123, group, d), randn(g, 271, 1, d), randn(g, 271, 1, d))
    starts = [ints(np.concatenate([[0], np.cumsum([n[i] for n in lens])]).tolist()) for i in range(2)]
    out = mxq.attention(q.to(DEV), k.to(DEV), v.to(DEV), *starts, window=(30, 0), sinks=2, scale=scale)
    attention_check(out, q, k, v, lens, 30, 0, 2, scale, "scale, ragged")


SCORED = [(3, 50, (-1, -1)), (70, 70, (-1, 0)), (2, 8000, (-1, -1)), (40, 300, (20, 0)), (1030, 6200, (-1, -1))]


def first_elements(q0, k0, nq, nk, heads, d, seed):
    """Queries and keys whose first elements alone make scores, and values: bf16."""
    q, k = torch.zeros(nq, heads, d), torch.zeros(nk, 1, d)
    q[..., 0], k[..., 0] = q0, k0
    return q.to(BF16), k.to(BF16), randn(gen(seed), nk, 1, d)


def paged_of(k, v, page=16):
    """The rows as the pages of one sequence: (cache, table)."""
    pages = -(-len(k) // page)
    held = []
    for t in (k, v):
        rows = torch.zeros(pages * page, *t.shape[1:], dtype=BF16)
        rows[:len(t)] = t
        held.append(rows.view(pages, page, *t.shape[1:]).transpose(1, 2).contiguous().to(DEV))
    return mxq.KvCache(*held), ints([list(range(pages))])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq, nk, window", SCORED)
def test_attention_scores_past_the_range(nq, nk, window, d):
    """Largest scores past 2^30 (in units of log2), finite ones and ones whose product with the scale is not: NaN, not the zeros of a
    row that sees nothing. Below it, rows of equal scores are means of values."""
    say("scores", nq, nk, window, d)
    heads = 64 if nq > 1000 else 2
    for q0, k0, scale, fine in ((2.0 ** 60, 2.0 ** 60, 1024.0, False), (2.0 ** 60, 2.0 ** 60, 1.0, False), (1.3e6, 1.1e6, 0.125, False),
                                (-(2.0 ** 60), 2.0 ** 60, 1.0, False), (-(2.0 ** 60), 2.0 ** 60, 1024.0, False),
                                (-1.3e6, 1.1e6, 0.125, False), (70000.0, 70000.0, 0.125, True), (-70000.0, 70000.0, 0.125, True)):
        q, k, v = first_elements(q0, k0, nq, nk, heads, d, nk)
        a = [t.to(DEV) for t in (q, k, v)]
        call = lambda: mxq.attention(*a, window=window, scale=scale)
        if fine:
            # (equal scores: the rounding of the exponent's argument is common to all weights and cancels)
            attention_check(call(), torch.zeros_like(q), k, v, [(nq, nk)], *window, 0, 1.0, "equal scores", heads=[0, heads - 1])
        else:
            assert torch.isnan(call()).all(), (q0, k0, scale)
            reported(call)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [3, 40, 5000])
def test_attention_paged_scores_past_the_range(n, d):
    say("scores, paged", n, d)
    for q0, k0, scale, fine in ((2.0 ** 60, 2.0 ** 60, 1024.0, False), (2.0 ** 60, 2.0 ** 60, 1.0, False), (1.3e6, 1.1e6, 0.125, False),
                                (-(2.0 ** 60), 2.0 ** 60, 1024.0, False), (-1.3e6, 1.1e6, 0.125, False),
                                (70000.0, 70000.0, 0.125, True), (-70000.0, 70000.0, 0.125, True)):
        q, k, v = first_elements(q0, k0, 1, n, 2, d, n)
        held, table = paged_of(k, v)
        call = lambda: mxq.attention_paged(q.to(DEV), held, table, ints([n]), scale=scale)
        if fine:
            attention_check(call(), torch.zeros_like(q), k, v, [(1, n)], -1, -1, 0, 1.0, "equal scores")
        else:
            assert torch.isnan(call()).all(), (q0, k0, scale)
            reported(call)


@pytest.mark.parametrize("nk, begin, end", [(300, 0, 70), (300, 130, 300), (9000, 0, 4100), (9000, 4000, 9000), (9000, 1, 9000)])
def test_attention_scores_far_below_the_others(nk, begin, end):
    """Keys whose scores are past the range below have no weight next to ordinary ones, wherever they lie."""
    say("far below", nk, begin, end)
    d, heads = 128, 2
    g = gen(nk + begin)
    q, k, v = randn(g, 3, heads, d), randn(g, nk, 1, d), randn(g, nk, 1, d)
    q[..., 0], k[..., 0] = 3e5, 0.0
    k[begin:end, :, 0] = -3e12
    keep = torch.tensor([j for j in range(nk) if not begin <= j < end])
    for window in ((-1, -1), (nk, 2)):
        out = mxq.attention(q.to(DEV), k.to(DEV), v.to(DEV), window=window)
        attention_check(out, q, k[keep], v[keep], [(3, len(keep))], -1, -1, 0, d ** -0.5, "below")
    held, table = paged_of(k, v)
    out = mxq.attention_paged(q[:1].to(DEV), held, table, ints([nk]))
    attention_check(out, q[:1], k[keep], v[keep], [(1, len(keep))], -1, -1, 0, d ** -0.5, "below, paged")


# ------------------------------------------------- numbers into an MXFP8 cache ----

@pytest.mark.parametrize("d, kv", [(64, 1), (128, 3)])
def test_mxfp8_cache_of_large_and_small_numbers(d, kv):
    """Blocks of every magnitude that bf16 has, the largest and subnormal ones among them: codes and scales as defined, and what
    attention reads of a single token is its value."""
    say("magnitudes", d, kv)
    g, m, page = gen(d), 262, 16
    v = torch.randn(m, 2 * kv, d, generator=g) * torch.exp2(torch.arange(m) - 134.0)[:, None, None].double()
    x = v.clamp(-3.3895e38, 3.3895e38).to(BF16)
    x[m - 1, :, 3], x[m - 2, :, 40] = 3.3895e38, -3.3895e38
    assert torch.isfinite(x).all()
    held = mxq.kv_cache(-(-m // page), kv, page, d, mxq.KV_MXFP8)
    for t in held:
        t.fill_(0x55)
    _, dense = mxq.rotary_qkv(x.view(m, -1).to(DEV), 0, kv, d, cache=held, slots=ints(list(range(m))))
    assert torch.equal(dense.cpu(), x[:, :kv])
    rows = []
    for codes, scales, value in ((held.k, held.k_scales, x[:, :kv]), (held.v, held.v_scales, x[:, kv:])):
        c, s = oracle.mxfp8_quantize(host(value))
        got = [t.cpu().transpose(1, 2).reshape(-1, kv, t.shape[3])[:m] for t in (codes, scales)]
        bits = np.where(c & 0x7F, 0xFF, 0x7F).astype(np.uint8)  # (a zero may have either sign)
        assert np.array_equal(got[0].numpy() & bits, c & bits)
        assert torch.equal(got[1], torch.from_numpy(s))
        rows.append(oracle.mxfp8_dequantize(c, s))
    # tokens at the start of their page, one to a sequence: the output is the value that the cache stands for, where bf16 has it
    # to all its bits (2^-126 on)
    first = list(range(0, m, page))
    q = torch.zeros(len(first), kv, d, dtype=BF16, device=DEV)
    out = host(mxq.attention_paged(q, held, ints([[i] for i in range(len(first))]), ints([1] * len(first))))
    want = rows[1][first]
    assert np.array_equal(np.where(np.abs(want) < 2.0 ** -126, 0, out), np.where(np.abs(want) < 2.0 ** -126, 0, want))


@pytest.mark.parametrize("d", [64, 128])
def test_caches_keep_infinities_and_nan(d):
    """What is not finite among keys and values shows in the same places of the output, whichever format the cache has."""
    say("not finite", d)
    kv, heads, m, nan, inf = 2, 4, 40, float("nan"), float("inf")
    base = randn(gen(d), m, (heads + 2 * kv) * d)
    base[:, :heads * d] = base[:, :heads * d].abs() + 0.1  # (an infinite key has a score of its sign)
    key, value = heads * d, (heads + kv) * d
    for name, places in (("nan key", [(7, key + 5, nan)]), ("-nan key", [(39, key + d + 33, -nan)]), ("nan value", [(7, value + 9, nan)]),
                         ("nan values", [(0, value, nan), (17, value + 2 * d - 1, nan)]), ("inf key", [(20, key + 1, inf)]),
                         ("inf values", [(3, value + 31, inf), (4, value + d + 32, -inf)])):
        x = base.clone()
        for r, c, what in places:
            x[r, c] = what
        seen = []
        for fmt in (mxq.KV_BF16, mxq.KV_MXFP8):
            held = mxq.kv_cache(3, kv, 16, d, fmt)
            q, _ = mxq.rotary_qkv(x.to(DEV), heads, kv, d, cache=held, slots=ints(list(range(m))), write_k=False)
            out = mxq.attention_paged(q[-1:], held, ints([[0, 1, 2]]), ints([m])).float().cpu()
            seen.append((torch.isnan(out), torch.isposinf(out), torch.isneginf(out)))
        for a, b in zip(*seen):
            assert torch.equal(a, b), name
        assert any(a.any() for a in seen[0]), name
        group = heads // kv  # only the heads that read the place
        for r, c, what in places:
            hk = (c - (key if c < value else value)) // d
            hit = torch.stack(seen[0]).any(0)[0]
            assert hit[hk * group:(hk + 1) * group].any(), name
        if "key" in name:
            assert hit[hk * group:(hk + 1) * group].all() and not hit[(1 - hk) * group:(2 - hk) * group].any(), name


# -------------------------------------------------------------- small norms ----

@pytest.mark.parametrize("norm", [mxq.ROTARY_NORM_ROW, mxq.ROTARY_NORM_HEAD])
@pytest.mark.parametrize("eps", [2.0 ** -126, 2.0 ** -120])
def test_rotary_norms_of_next_to_nothing(norm, eps):
    """Rows of zeros and rows whose squares are subnormal, the smallest eps."""
    say("small norms", norm, eps)
    m, heads, kv, d = 40, 4, 2, 64
    x = randn(gen(1), m, (heads + 2 * kv) * d).double() * torch.exp2(-torch.arange(m).double() - 50.0)[:, None]
    x = x.to(BF16)
    x[5] = 0
    q, k = mxq.rotary_qkv(x.to(DEV), heads, kv, d, norm=norm, eps=eps)
    want = rotary_want(x, heads, kv, d, torch.zeros(0, dtype=torch.float64), [], None, [torch.ones(d * (heads if norm == 1 else 1)),
                                                                                         torch.ones(d * (kv if norm == 1 else 1))],
                       norm, False, eps)
    rotary_within(q, want[0], "q")
    rotary_within(k, want[1], "k")
    assert not q[5].any() and not k[5].any()
