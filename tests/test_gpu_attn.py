"""GPU tests of the attention half of a block (include/mxq_attention.h) against its definitions in float64 on the CPU.

Tolerances, with u = 2^-24 (half an fp32 step) and 2^-8 (half a bf16 step) relative to the value:

* rotary: a sum of squares passes at most 64 + 10 additions in depth, so with square root, division and the products after it a
  normed value is off by less than 64 u; sine and cosine (of an angle reduced in 64 bits, then rounded to fp32 revolutions) by
  less than 8 u. A rotated element is thus off by less than 128 u = 2^-17 of |a| + |b|, and by one rounding to bf16.
* attention: a score is an fp32 sum of D products, off by at most 2 D u of sum |q k|; the exponent's argument adds 4 u of the
  largest score, and the running maximum's corrections as much again per key tile that raises it, which is bounded by the
  number of tiles. A weight is then off by d = (2 D + 8 + 4 tiles) u scale sum |q k| + 2^-20 (exponential, sums) relative, and
  by 2^-8 where it is rounded to bf16 before its product with v; numerator and denominator each, so the output is off by
  (2 d + 2^-8) sum w |v| and one rounding to bf16.
"""

import sys

import numpy as np
import pytest
import torch

import mx_bit_quantized_amd as mxq
import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
DEV = "cuda:0"
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    mxq.lib()
    yield
    torch.cuda.synchronize()


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=g)).to(BF16)


def ints(v):
    return torch.tensor(v, dtype=I32, device=DEV)


def host(t):
    return t.detach().cpu().double().numpy()


def within(got, want, tol, what):
    got = host(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got - want) - tol
    assert off.max(initial=-1.0) <= 0, f"{what}: {np.argwhere(off > 0)[:4].tolist()} off by {off.max()} more than allowed"


# ------------------------------------------------------------------ plan ----

PLANS = [  # cached, added, width, free, page, tokens
    ([0], [1], 1, 1, 16, 1),
    ([16], [1], 3, 2, 16, 4),
    ([15, 0, 33], [1, 0, 70], 8, 9, 16, 80),
    ([5, 31, 32, 64], [0, 0, 0, 0], 4, 0, 32, 3),
    ([100, 3], [40, 500], 9, 40, 64, 600),
    ([40, 40], [30, 90], 4, 3, 16, 140),       # the list is used up, the table too narrow
    ([200, 0], [5, 5], 2, 9, 16, 10),          # cached past the table
    ([1, 2, 3], [10, 10, 10], 4, 8, 16, 12),   # more tokens than places
    ([-4, 7], [3, -2], 4, 8, 16, 5),
    ([], [], 3, 2, 16, 5),
    ([7] * 300, [1] * 300, 2, 10, 1024, 301),
    ([i % 50 for i in range(4096)], [i % 3 for i in range(4096)], 4, 4096, 16, 4100),
]


def table_of(cached, width, page, free, seed):
    pages = np.random.default_rng(seed).permutation(sum(-(-max(c, 0) // page) for c in cached) + free + 3).tolist()
    table = np.full((len(cached), width), -1, np.int64)
    for r, c in enumerate(cached):
        for col in range(min(-(-max(c, 0) // page), width)):
            table[r, col] = pages.pop()
    return table, pages[:free]


@pytest.mark.parametrize("case", range(len(PLANS)))
def test_page_plan(case):
    cached, added, width, free, page, tokens = PLANS[case]
    table, pages = table_of(cached, width, page, free, case)
    say("plan", case, len(cached), tokens)
    t = torch.tensor(table, dtype=I32, device=DEV).view(len(cached), width)
    got = mxq.page_plan(ints(cached), ints(added), t, ints(pages), page, tokens)
    want = oracle.page_plan(cached, added, table, pages, page, tokens)
    for name, g, w in zip(mxq.PagePlan._fields, got, want):
        assert g.cpu().tolist() == list(w), name
    assert np.array_equal(t.cpu().numpy(), want[5])


def test_page_plan_missing_old_page():
    table = np.array([[-1, -1, -1]])
    t = torch.tensor(table, dtype=I32, device=DEV)
    got = mxq.page_plan(ints([5]), ints([20]), t, ints([4]), 16, 20)
    want = oracle.page_plan([5], [20], table, [4], 16, 20)
    assert [g.cpu().tolist() for g in got] == [list(w) for w in want[:5]] and np.array_equal(t.cpu().numpy(), want[5])


# ---------------------------------------------------------------- rotary ----

def rotary_case(m, heads, kv, d, pairs, axes, norm, seed, far=False, padding=0):
    g = gen(seed)
    x = randn(g, m, (heads + 2 * kv) * d + padding, scale=2.0)
    counts = [pairs - (axes - 1) * (pairs // 3)] + [pairs // 3] * (axes - 1) if pairs else []
    freqs, axis = mxq.rotary_frequencies(counts, 10000.0, device="cpu")
    pos = torch.randint(-50, 50, (axes, m), generator=g) if not far else torch.randint(2 ** 30, 2 ** 31 - 1, (axes, m), generator=g)
    of = (heads * d, kv * d) if norm == 1 else (d, d)
    weights = [None if norm == 0 else (1 + 0.2 * torch.randn(n, generator=g)).to(BF16) for n in of]
    return x, freqs, axis, pos.to(I32), weights


def rotary_want(x, heads, kv, d, freqs, axis, pos, weights, norm, interleaved, eps=1e-6):
    """(want, |a| + |b|) of q and of k, float64 [m, heads, d]."""
    m = x.shape[0]
    rows = host(x)[:, :(heads + 2 * kv) * d].reshape(m, -1, d)
    angle = (pos.double()[axis.long()] * freqs[:, None]).numpy().T if len(axis) else np.zeros((m, 0))
    out = []
    for part, w in ((rows[:, :heads], weights[0]), (rows[:, heads:heads + kv], weights[1])):
        if norm == 1 and part.size:
            part = oracle.rms_norm(part.reshape(m, -1), host(w), eps).reshape(part.shape)
        elif norm == 2:
            part = oracle.rms_norm(part, host(w), eps)
        a = angle[:, None, :]
        size = oracle.rotate(np.abs(part), np.full(a.shape, np.pi / 4), interleaved) * np.sqrt(2)
        pairs = a.shape[-1]
        # |a| + |b| of a pair is sqrt(2) times the sine part of its turn by 45 degrees
        if pairs:
            if interleaved:
                size[..., 0:2 * pairs:2] = size[..., 1:2 * pairs:2]
            else:
                size[..., :pairs] = size[..., pairs:2 * pairs]
        size[..., 2 * pairs:] = np.abs(part[..., 2 * pairs:])
        out.append((oracle.rotate(part, a, interleaved), size))
    return out


def rotary_within(got, want, what):
    value, size = want
    slack = 2.0 ** -17 * size
    within(got, value, BF * (np.abs(value) + slack) + slack, what)


ROTARY = [  # m, heads, kv, d, pairs, axes, norm, interleaved
    (1, 1, 1, 64, 32, 1, 0, False),
    (1, 40, 8, 128, 64, 1, 2, False),
    (3, 5, 5, 128, 64, 3, 1, True),
    (37, 12, 4, 64, 16, 3, 2, True),
    (37, 12, 4, 64, 16, 2, 2, False),
    (70, 3, 1, 128, 24, 1, 1, False),
    (9, 7, 7, 128, 8, 1, 2, True),
    (5, 0, 4, 128, 64, 1, 1, False),
    (5, 6, 0, 64, 32, 1, 1, True),
    (11, 2, 2, 128, 0, 1, 1, False),
    (4, 128, 128, 128, 64, 3, 1, True),   # more units than a workgroup has threads
    (4, 170, 170, 128, 64, 1, 2, False),
    (2051, 16, 1, 64, 32, 3, 2, True),
]


@pytest.mark.parametrize("m, heads, kv, d, pairs, axes, norm, interleaved", ROTARY)
@pytest.mark.parametrize("cache", [None, mxq.KV_BF16, mxq.KV_MXFP8])
def test_rotary_qkv(m, heads, kv, d, pairs, axes, norm, interleaved, cache):
    if cache is not None and kv == 0:
        pytest.skip("a row without keys has nothing to cache")
    say("rotary", m, heads, kv, d, pairs, axes, norm, interleaved, cache)
    x, freqs, axis, pos, weights = rotary_case(m, heads, kv, d, pairs, axes, norm, m + heads)
    page, pages = 16, m // 16 + 3
    dev = lambda t: None if t is None else t.to(DEV)
    turn = dict(positions=dev(pos), freqs=dev(freqs), axis=dev(axis)) if pairs else {}
    w = [dev(t) for t in weights]
    if heads == 0:
        w[0] = None
    if kv == 0:
        w[1] = None
    held = slots = None
    if cache is not None:
        held = mxq.kv_cache(pages, kv, page, d, cache)
        for t in held:
            if t is not None:
                t.fill_(3)
        slots = torch.randperm(pages * page, generator=gen(m))[:m].to(I32)
        slots[::5] = -1
        slots[2::7] = pages * page + 4  # outside the cache
    q, k = mxq.rotary_qkv(dev(x), heads, kv, d, **turn, interleaved=interleaved, norm=norm, q_weight=w[0], k_weight=w[1],
                          cache=held, slots=dev(slots))
    want = rotary_want(x, heads, kv, d, freqs, axis, pos, weights, norm, interleaved)
    if heads:
        rotary_within(q, want[0], "q")
    else:
        assert q is None
    if kv:
        rotary_within(k, want[1], "k")
    else:
        assert k is None
    if cache is None:
        return
    # the cache holds the dense k and v bit for bit (or their codes), other slots stay
    v = x[:, (heads + kv) * d:(heads + 2 * kv) * d].view(m, kv, d)
    kept = [(int(s), r) for r, s in enumerate(slots.tolist()) if 0 <= s < pages * page]
    for dense, codes, scales in ((k.cpu(), held.k.cpu(), held.k_scales), (v, held.v.cpu(), held.v_scales)):
        flat = codes.transpose(1, 2).reshape(pages * page, kv, d).clone()
        expect = torch.full_like(flat, 3)
        for s, r in kept:
            expect[s] = dense[r] if cache == mxq.KV_BF16 else torch.from_numpy(oracle.mxfp8_quantize(host(dense[r]))[0])
        assert torch.equal(flat, expect)
        if cache == mxq.KV_MXFP8:
            flat = scales.cpu().transpose(1, 2).reshape(pages * page, kv, d // 32)
            expect = torch.full_like(flat, 3)
            for s, r in kept:
                expect[s] = torch.from_numpy(oracle.mxfp8_quantize(host(dense[r]))[1])
            assert torch.equal(flat, expect)
    q2, k2 = mxq.rotary_qkv(dev(x), heads, kv, d, **turn, interleaved=interleaved, norm=norm, q_weight=w[0], k_weight=w[1],
                            cache=held, slots=dev(slots), write_k=False)
    assert k2 is None and (q is None or torch.equal(q, q2))


def test_rotary_far_positions():
    """Angles of up to 2^31 radians."""
    m, heads, kv, d = 16, 2, 1, 128
    x, freqs, axis, pos, weights = rotary_case(m, heads, kv, d, 64, 3, 2, 5, far=True)
    q, k = mxq.rotary_qkv(x.to(DEV), heads, kv, d, pos.to(DEV), freqs.to(DEV), axis.to(DEV), norm=2, q_weight=weights[0].to(DEV),
                          k_weight=weights[1].to(DEV))
    want = rotary_want(x, heads, kv, d, freqs, axis, pos, weights, 2, False)
    rotary_within(q, want[0], "q")
    rotary_within(k, want[1], "k")


def test_rotary_strides_in_place_and_defaults():
    m, heads, kv, d = 21, 6, 2, 64
    x, freqs, axis, pos, weights = rotary_case(m, heads, kv, d, 32, 1, 2, 8, padding=64)
    wide = x.to(DEV)
    rows = wide[:, :(heads + 2 * kv) * d]  # rows with a stride
    a = dict(freqs=freqs.to(DEV), norm=mxq.ROTARY_NORM_HEAD, q_weight=weights[0].to(DEV), k_weight=weights[1].to(DEV))
    q, k = mxq.rotary_qkv(rows, heads, kv, d, pos[0].to(DEV), **a)  # positions of one axis, no axis map
    want = rotary_want(x, heads, kv, d, freqs, axis, pos, weights, 2, False)
    rotary_within(q, want[0], "q")
    rotary_within(k, want[1], "k")
    assert torch.equal(wide, x.to(DEV))
    vq = rows[:, :heads * d].view(m, heads, d)
    vk = rows[:, heads * d:(heads + kv) * d].view(m, kv, d)
    q2, k2 = mxq.rotary_qkv(rows, heads, kv, d, pos[0].to(DEV), **a, q=vq, k=vk)
    assert q2 is vq and torch.equal(vq, q) and torch.equal(vk, k)
    assert torch.equal(wide[:, (heads + kv) * d:].cpu(), x[:, (heads + kv) * d:])


def test_rotary_axes_outside():
    """Pairs on an axis that the positions do not have are not turned."""
    m, heads, d = 4, 2, 64
    x = randn(gen(1), m, heads * d)
    freqs = torch.ones(32, dtype=torch.float64, device=DEV)
    axis = torch.tensor([0, 5, -1, 1] * 8, dtype=I32, device=DEV)
    q, _ = mxq.rotary_qkv(x.to(DEV), heads, 0, d, torch.full((2, m), 3, dtype=I32, device=DEV), freqs, axis, interleaved=True)
    y, z = x.view(m, heads, 32, 2), q.cpu().view(m, heads, 32, 2)
    for p, a in enumerate(axis.tolist()):
        assert torch.equal(y[:, :, p], z[:, :, p]) == (a not in (0, 1))


# ------------------------------------------------------------- attention ----

def attention_check(out, q, k, v, lens, left, right, sinks, scale, what, heads=None):
    """Every row of every sequence (or of some heads) against the definition; lens: (queries, keys) of each sequence."""
    q, k, v = host(q), host(k), host(v)
    mq, h, d = q.shape
    group = h // k.shape[1]
    q0 = k0 = 0
    want, tol = np.zeros(q.shape), np.zeros(q.shape)
    for nq, nk in lens:
        for head in range(h) if heads is None else heads:
            g = head // group
            o, mean, top = oracle.attention_rows(q[q0:q0 + nq, head], k[k0:k0 + nk, g], v[k0:k0 + nk, g], nk - nq, left, right, sinks,
                                                 scale)
            off = (2 * d + 8 + 4 * (nk // 64 + 2)) * U * top[:, None] + 2.0 ** -20
            slack = (2 * off + BF) * mean
            want[q0:q0 + nq, head], tol[q0:q0 + nq, head] = o, BF * (np.abs(o) + slack) + slack
        q0, k0 = q0 + nq, k0 + nk
    got = host(out)[:q0]
    pick = slice(None) if heads is None else list(heads)
    within(got[:, pick], want[:q0][:, pick], tol[:q0][:, pick], what)


ATTENTION = [  # lens, heads, kv, d, left, right, sinks
    ([(1, 1)], 1, 1, 64, -1, -1, 0),
    ([(1, 300)], 8, 1, 128, -1, 0, 0),
    ([(64, 64)], 2, 2, 128, -1, 0, 0),
    ([(65, 63)], 2, 1, 64, -1, 0, 0),              # rows ahead of the first key
    ([(33, 129)], 3, 3, 128, -1, -1, 0),
    ([(300, 300)], 5, 1, 128, -1, 0, 0),
    ([(257, 513)], 4, 2, 64, 40, 0, 0),
    ([(257, 513)], 4, 2, 128, 40, 0, 5),
    ([(200, 700)], 2, 2, 64, 100, 0, 130),
    ([(200, 700)], 2, 2, 128, 63, 64, 3),
    ([(130, 130)], 2, 1, 128, 0, 0, 0),            # each token sees itself
    ([(130, 130)], 2, 1, 64, -1, 7, 0),
    ([(0, 5), (7, 0), (1, 1), (3, 200), (150, 150), (0, 0), (2, 1)], 4, 2, 128, -1, 0, 0),
    ([(40, 90), (90, 40), (13, 13), (260, 400)], 6, 2, 64, 30, 2, 4),
    ([(1, 2000), (1, 3), (2, 1000)], 10, 2, 128, 500, 0, 4),
    ([(17, 64 * 40 + 5)], 16, 1, 64, -1, 0, 0),    # few rows, a long axis: joined from parts
    ([(5, 4096)], 3, 3, 128, -1, -1, 0),
    ([(5, 4096)], 3, 3, 128, 1000, 0, 70),
    ([(300, 6300)], 2, 1, 128, -1, 0, 0),          # long axes of heads of 128
    ([(513, 6145)], 1, 1, 128, -1, -1, 0),
    ([(70, 7000), (200, 6500), (0, 20), (3, 13000)], 3, 1, 128, -1, 5, 0),
    ([(130, 12700)], 4, 2, 128, 6100, 200, 3),
]


@pytest.mark.parametrize("lens, heads, kv, d, left, right, sinks", ATTENTION)
def test_attention(lens, heads, kv, d, left, right, sinks):
    say("attention", lens, heads, kv, d, left, right, sinks)
    g = gen(len(lens) * 1000 + heads)
    mq, mk = sum(n for n, _ in lens), sum(n for _, n in lens)
    q, k, v = randn(g, mq, heads, d, scale=1.5), randn(g, mk, kv, d, scale=1.5), randn(g, mk, kv, d)
    starts = [ints(np.concatenate([[0], np.cumsum([n[i] for n in lens])]).tolist()) for i in range(2)]
    a = [t.to(DEV) for t in (q, k, v)]
    out = mxq.attention(*a, *starts, window=(left, right), sinks=sinks)
    attention_check(out, q, k, v, lens, left, right, sinks, d ** -0.5, "attention")
    assert torch.equal(out, mxq.attention(*a, *starts, window=(left, right), sinks=sinks))
    if len(lens) == 1:
        assert torch.equal(out, mxq.attention(*a, window=(left, right), sinks=sinks))


def test_attention_scale_and_views():
    """Views of one stacked projection, an output with a row stride, a scale of its own."""
    m, heads, kv, d = 150, 4, 2, 64
    x = randn(gen(3), m, (heads + 2 * kv) * d + 8).to(DEV)
    q = x[:, :heads * d].view(m, heads, d)
    k = x[:, heads * d:(heads + kv) * d].view(m, kv, d)
    v = x[:, (heads + kv) * d:(heads + 2 * kv) * d].view(m, kv, d)
    buf = torch.full((m, heads * d + 64), 7.0, dtype=BF16, device=DEV)
    out = buf[:, :heads * d].view(m, heads, d)
    assert mxq.attention(q, k, v, window=(-1, 0), scale=0.3, out=out) is out
    attention_check(out, q, k, v, [(m, m)], -1, 0, 0, 0.3, "views")
    assert (buf[:, heads * d:] == 7).all()


def test_attention_rows_behind_the_last_sequence():
    heads, kv, d = 4, 2, 128
    lens = [(20, 70), (50, 30)]
    g = gen(4)
    q, k, v = randn(g, 100, heads, d), randn(g, 140, kv, d), randn(g, 140, kv, d)
    q[70:], k[100:], v[100:] = float("nan"), float("nan"), float("inf")
    for n, keys in ((0, 140), (1, 140)):
        out = torch.full((100, heads, d), 5.0, dtype=BF16, device=DEV)
        mxq.attention(q.to(DEV), k.to(DEV), v.to(DEV), ints([0, 20, 70]), ints([0, 70, 100]), window=(-1, 0 if n else -1), out=out)
        attention_check(out, q, k, v, lens, -1, 0 if n else -1, 0, d ** -0.5, "padded")
        assert (out[70:] == 5).all()


def test_attention_large_scores():
    """Scores far above the range of an exponential, and rows of equal ones."""
    m, d = 90, 64
    q, k, v = randn(gen(5), m, 2, d, scale=30.0), randn(gen(6), m, 2, d, scale=30.0), randn(gen(7), m, 2, d)
    out = mxq.attention(q.to(DEV), k.to(DEV), v.to(DEV), window=(-1, 0))
    attention_check(out, q, k, v, [(m, m)], -1, 0, 0, d ** -0.5, "large")
    z = torch.zeros_like(q)
    out = mxq.attention(z.to(DEV), k.to(DEV), v.to(DEV))
    attention_check(out, z, k, v, [(m, m)], -1, -1, 0, d ** -0.5, "equal")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("left, right, sinks, nk", [(-1, 0, 0, 150), (40, 0, 3, 300), (20, 30, 0, 300), (-1, 0, 0, 4100)])
def test_attention_hidden_places_hold_anything(d, left, right, sinks, nk):
    """Infinities and NaN among keys and values reach the rows that see them and no others."""
    nq, heads, kv = 150, 2, 1
    say("hidden", d, left, right, sinks, nk)
    g = gen(d)
    q, k, v = randn(g, nq, heads, d), randn(g, nk, kv, d), randn(g, nk, kv, d)
    first = nk - nq
    nan, inf = float("nan"), float("inf")
    k[nk - 9, 0, 5], k[first + 70, 0, 1] = nan, inf
    v[nk - 30, 0, 3], v[nk - 31, 0, 4], v[nk - 31, 0, d - 1], v[nk - 7, 0, 17] = nan, inf, -inf, inf
    v[first + 31, 0, 33] = -inf
    out = host(mxq.attention(q.to(DEV), k.to(DEV), v.to(DEV), window=(left, right), sinks=sinks))
    clean = 0
    for h in range(heads):
        with np.errstate(all="ignore"):
            o, mean, top = oracle.attention_rows(host(q)[:, h], host(k)[:, 0], host(v)[:, 0], first, left, right, sinks, d ** -0.5)
        # a score of +inf leaves no finite weight: the definition's row is NaN
        for i in range(nq):
            if np.isnan(o[i]).all():
                assert np.isnan(out[i, h]).all(), i
                continue
            fine = np.isfinite(o[i])
            clean += fine.all()
            assert np.array_equal(np.isnan(o[i]), np.isnan(out[i, h])) and np.array_equal(o[i][~fine], out[i, h][~fine], equal_nan=True), i
            off = (2 * (2 * d + 8 + 4 * (nk // 64 + 2)) * U * top[i] + 2.0 ** -19 + BF) * mean[i][fine]
            assert (np.abs(out[i, h][fine] - o[i][fine]) <= BF * (np.abs(o[i][fine]) + off) + off).all(), i
    assert clean > 20


# ----------------------------------------------------------------- paged ----

def paged_case(lengths, kv, d, page, fmt, seed, width=None, spare=3):
    """(cache on the GPU, table, keys and values [tokens of b] as the cache holds them)."""
    g = gen(seed)
    counts = [-(-n // page) for n in lengths]
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=g).tolist()
    width = width or max(counts + [1]) + 1
    table = np.full((len(lengths), width), -1, np.int64)
    kc, vc = randn(g, pages, kv, page, d, scale=1.5), randn(g, pages, kv, page, d)
    if fmt == mxq.KV_MXFP8:
        parts = [oracle.mxfp8_quantize(host(t)) for t in (kc, vc)]
        held = mxq.KvCache(*(torch.from_numpy(np.ascontiguousarray(p[i])).to(DEV) for i in range(2) for p in parts))
        kc, vc = (torch.from_numpy(oracle.mxfp8_dequantize(*p)).to(BF16) for p in parts)
    else:
        held = mxq.KvCache(kc.to(DEV), vc.to(DEV))
    rows = []
    for b, n in enumerate(lengths):
        ids = [order.pop() for _ in range(counts[b])]
        table[b, :len(ids)] = ids[:width]
        rows.append([t[ids].transpose(1, 2).reshape(-1, kv, d)[:n] for t in (kc, vc)] if n else [kc[:0, :, 0], vc[:0, :, 0]])
    return held, torch.tensor(table, dtype=I32, device=DEV), rows


def paged_check(out, q, rows, lengths, left, sinks, scale, what):
    for b, n in enumerate(lengths):
        attention_check(out[b:b + 1], q[b:b + 1], *rows[b], [(1, n)], left, 0, sinks, scale, f"{what} {b}")


PAGED = [  # lengths, heads, kv, d, page, left, sinks
    ([1], 1, 1, 64, 16, -1, 0),
    ([17], 8, 1, 128, 16, -1, 0),
    ([0, 1, 15, 16, 17, 0, 33], 4, 2, 128, 16, -1, 0),
    ([5000], 40, 8, 128, 16, -1, 0),
    ([3000, 1, 2, 700], 16, 2, 64, 64, -1, 0),
    ([900, 40, 2000], 40, 2, 128, 32, 100, 4),      # 20 heads of a key head
    ([900, 40, 2000, 130], 6, 6, 64, 16, 127, 70),
    ([1500, 3], 33, 1, 128, 1024, -1, 0),
    ([129, 128, 127], 12, 4, 64, 128, 0, 0),        # only the new token itself
    ([65] * 70, 5, 5, 128, 64, -1, 0),
    ([300, 7, 256], 10, 2, 128, 256, 63, 16),
]


@pytest.mark.parametrize("lengths, heads, kv, d, page, left, sinks", PAGED)
@pytest.mark.parametrize("fmt", [mxq.KV_BF16, mxq.KV_MXFP8])
def test_attention_paged(lengths, heads, kv, d, page, left, sinks, fmt):
    say("paged", lengths[:8], heads, kv, d, page, left, sinks, fmt)
    held, table, rows = paged_case(lengths, kv, d, page, fmt, len(lengths) + d)
    q = randn(gen(heads), len(lengths), heads, d, scale=1.5)
    a = (q.to(DEV), held, table, ints(lengths))
    out = mxq.attention_paged(*a, window=left, sinks=sinks)
    paged_check(out, q, rows, lengths, left, sinks, d ** -0.5, "paged")
    assert torch.equal(out, mxq.attention_paged(*a, window=left, sinks=sinks))


@pytest.mark.parametrize("fmt", [mxq.KV_BF16, mxq.KV_MXFP8])
def test_attention_paged_what_pages_hold_elsewhere(fmt):
    """Places past the length, before the window and on pages that the cache does not have may hold anything."""
    lengths, kv, d, page, heads, left, sinks = [70, 130, 90, 200], 2, 64, 32, 4, 50, 3
    held, table, rows = paged_case(lengths, kv, d, page, fmt, 9)
    q = randn(gen(10), len(lengths), heads, d)
    for b, n in enumerate(lengths):
        for col in range(-(-n // page)):
            for at in range(page):
                j = col * page + at
                if j < n and (j >= n - 1 - left or j < sinks):
                    continue
                p = table[b, col].item()
                if fmt == mxq.KV_BF16:
                    held.k[p, :, at], held.v[p, :, at] = float("nan"), float("inf") if j % 2 else float("nan")
                else:
                    held.k[p, :, at], held.v[p, :, at], held.k_scales[p, :, at], held.v_scales[p, :, at] = 0x7F, 0xFF, 255, 255
    out = mxq.attention_paged(q.to(DEV), held, table, ints(lengths), window=left, sinks=sinks)
    paged_check(out, q, rows, lengths, left, sinks, d ** -0.5, "elsewhere")
    # a lost page: its keys are not visible
    held, table, rows = paged_case(lengths, kv, d, page, fmt, 11)
    table[1, 2], table[3, 0], table[2, 1] = -1, 10 ** 6, -7
    out = mxq.attention_paged(q.to(DEV), held, table, ints(lengths))
    lost = {1: 2, 3: 0, 2: 1}
    for b, n in enumerate(lengths):
        k, v = rows[b]
        if b in lost:
            keep = torch.tensor([j for j in range(n) if j // page != lost[b]])
            k, v = k[keep], v[keep]
        attention_check(out[b:b + 1], q[b:b + 1], k, v, [(1, len(k))], -1, -1, 0, d ** -0.5, f"lost page {b}")


def test_attention_paged_lengths_past_the_table():
    """Keys behind the table are not visible; the query's position is the length's."""
    held, table, rows = paged_case([64, 64], 1, 64, 16, mxq.KV_BF16, 12, width=4)
    q = randn(gen(13), 2, 2, 64)
    out = mxq.attention_paged(q.to(DEV), held, table, ints([70, 200]), window=20)
    for b, full in enumerate((70, 200)):
        lo = full - 1 - 20
        attention_check(out[b:b + 1], q[b:b + 1], rows[b][0][lo:], rows[b][1][lo:], [(1, max(0, 64 - lo))], -1, -1, 0, 0.125, f"past {b}")
    assert not out[1].any()
    out = mxq.attention_paged(q.to(DEV), held, table, ints([-5, 64]), scale=0.4)
    assert not out[0].any()
    attention_check(out[1:], q[1:], *rows[1], [(1, 64)], -1, 0, 0, 0.4, "scale")
