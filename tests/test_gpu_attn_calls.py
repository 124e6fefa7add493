"""GPU tests of calls of the attention half that its documents allow and that few programs make: nothing to attend, the most heads,
one tensor in two places, sequences that leave rows out on either side, and device values that are wrong (they give wrong results,
never an access outside the buffers). Tolerances: those of test_gpu_attn.py."""

import numpy as np
import pytest
import torch

import mx_bit_quantized_amd as mxq
from test_gpu_attn import (BF16, DEV, I32, attention_check, gen, host, ints, paged_case, paged_check, randn, rotary_case, rotary_want,
                           rotary_within, say)

pytestmark = pytest.mark.gpu


def starts_of(lens, first=(0, 0)):
    return [ints((first[i] + np.concatenate([[0], np.cumsum([n[i] for n in lens])])).tolist()) for i in range(2)]


# ------------------------------------------------------------- attention ----

def test_attention_of_nothing():
    say("nothing")
    heads, kv, d = 4, 2, 64
    q, none, no_q = (torch.randn(n, h, d, device=DEV).to(BF16) for n, h in ((200, heads), (0, kv), (0, heads)))
    for window in ((-1, -1), (-1, 0), (3, 3)):
        assert not mxq.attention(q, none, none, window=window).any()
        assert not mxq.attention(q, none, none, ints([0, 50, 200]), ints([0, 0, 0]), window=window).any()
        assert mxq.attention(no_q, q[:, :kv].contiguous(), q[:, :kv].contiguous(), window=window).shape == (0, heads, d)
    k = torch.randn(9, kv, d, device=DEV).to(BF16)
    out = torch.full_like(q, 3.0)
    mxq.attention(q, k, k, ints([0]), ints([0]), out=out)  # no sequences
    mxq.attention(q, k, k, ints([7, 7]), ints([0, 9]), out=out)  # one without queries
    assert (out == 3).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads, kv, nq, nk", [(1024, 1, 3, 70), (1024, 1024, 2, 33), (1024, 8, 40, 20), (960, 3, 5, 900)])
def test_attention_most_heads(heads, kv, nq, nk, d):
    say("most heads", heads, kv, nq, nk, d)
    g = gen(heads + kv)
    q, k, v = randn(g, nq, heads, d, scale=1.5), randn(g, nk, kv, d, scale=1.5), randn(g, nk, kv, d)
    some = sorted({0, heads // kv - 1, heads // 2, heads - 1})
    out = mxq.attention(*(t.to(DEV) for t in (q, k, v)), window=(-1, 0))
    attention_check(out, q, k, v, [(nq, nk)], -1, 0, 0, d ** -0.5, "most heads", heads=some)
    held, table, rows = paged_case([nk, 1], kv, d, 32, mxq.KV_BF16, nk)
    out = mxq.attention_paged(q[:2].to(DEV), held, table, ints([nk, 1]))
    for b, n in enumerate((nk, 1)):
        attention_check(out[b:b + 1], q[b:b + 1], *rows[b], [(1, n)], -1, 0, 0, d ** -0.5, "most heads, paged", heads=some)


def test_attention_one_tensor_for_keys_and_values():
    say("k is v")
    g, n, d = gen(1), 300, 128
    x = randn(g, n, 4, d)
    t = x.to(DEV)
    attention_check(mxq.attention(t, t, t, window=(50, 0)), x, x, x, [(n, n)], 50, 0, 0, d ** -0.5, "one tensor")


@pytest.mark.parametrize("lens, first, heads, kv, d", [([(70, 100), (5, 5), (130, 200)], (13, 29), 4, 2, 128),
                                                       ([(3, 9000), (2, 100)], (4, 700), 4, 1, 64)])
def test_attention_rows_outside_the_sequences(lens, first, heads, kv, d):
    """Sequences that begin behind the first row and end before the last one, of q and of k."""
    say("outside", lens, first)
    g = gen(sum(first))
    mq, mk = (sum(n[i] for n in lens) for i in range(2))
    q, k, v = randn(g, first[0] + mq + 6, heads, d), randn(g, first[1] + mk + 50, kv, d), randn(g, first[1] + mk + 50, kv, d)
    for t, at, n in ((q, first[0], mq), (k, first[1], mk), (v, first[1], mk)):
        t[:at], t[at + n:] = float("nan"), float("inf")
    out = torch.full(q.shape, 9.0, dtype=BF16, device=DEV)
    mxq.attention(*(t.to(DEV) for t in (q, k, v)), *starts_of(lens, first), window=(-1, 0), out=out)
    assert (out[:first[0]] == 9).all() and (out[first[0] + mq:] == 9).all()
    inner = [t[at:at + n] for t, at, n in ((q, first[0], mq), (k, first[1], mk), (v, first[1], mk))]
    attention_check(out[first[0]:first[0] + mq], *inner, lens, -1, 0, 0, d ** -0.5, "outside")


def test_attention_thousands_of_sequences():
    say("thousands")
    g, heads, kv, d = gen(2), 2, 1, 64
    lens = [(i * 7 % 4, i * 13 % 40) for i in range(5000)]
    mq, mk = (sum(n[i] for n in lens) for i in range(2))
    q, k, v = randn(g, mq, heads, d), randn(g, mk, kv, d), randn(g, mk, kv, d)
    out = mxq.attention(*(t.to(DEV) for t in (q, k, v)), *starts_of(lens), window=(20, 0), sinks=1)
    attention_check(out, q, k, v, lens, 20, 0, 1, d ** -0.5, "thousands", heads=[1])


@pytest.mark.parametrize("d, parts", [(64, False), (128, False), (64, True), (128, True)])
def test_attention_wrong_starts(d, parts):
    """Starts that decrease, lie before the first row or past the last one: guard rows on both sides of out stay, and the next call
    is right."""
    say("wrong starts", d, parts)
    g, heads, kv, mq, mk = gen(3), 4, 2, (7 if parts else 150), (9000 if parts else 200)
    q, k, v = (randn(g, m, h, d).to(DEV) for m, h in ((mq, heads), (mk, kv), (mk, kv)))
    buf = torch.full((mq + 600, heads, d), 4.0, dtype=BF16, device=DEV)
    out = buf[300:300 + mq]
    big = (1 << 31) - 1
    for sq, sk in (([0, mq // 2, 3, mq], [0, 100, 40, mk]), ([-5, mq // 3, big], [-big, 9, big]), ([mq, 3, 0], [mk, 5, 0]),
                   ([big, -big, big, 0], [big, 0, -7, big]), ([0, mq], [50, mk + 999])):
        mxq.attention(q, k, v, ints(sq), ints(sk), window=(-1, 0), out=out)
        torch.cuda.synchronize()
        assert (buf[:300] == 4).all() and (buf[300 + mq:] == 4).all(), (sq, sk)
    out = mxq.attention(q, k, v, ints([0, mq]), ints([0, mk]), window=(-1, 0))
    attention_check(out, q, k, v, [(mq, mk)], -1, 0, 0, d ** -0.5, "after wrong starts")


# ----------------------------------------------------------------- paged ----

def test_attention_paged_output_with_a_stride():
    say("paged views")
    lengths, heads, kv, d = [50, 0, 17, 300], 6, 2, 64
    held, table, rows = paged_case(lengths, kv, d, 16, mxq.KV_BF16, 3)
    wide = randn(gen(4), 4, (heads + 3) * d)
    buf = torch.full((4, heads * d + 24), 7.0, dtype=BF16, device=DEV)
    out = buf[:, 8:8 + heads * d].view(4, heads, d)
    q = wide.to(DEV)[:, d:(heads + 1) * d].view(4, heads, d)
    assert mxq.attention_paged(q, held, table, ints(lengths), out=out) is out
    paged_check(out, q.cpu(), rows, lengths, -1, 0, d ** -0.5, "views")
    assert (buf[:, :8] == 7).all() and (buf[:, 8 + heads * d:] == 7).all()


def test_attention_paged_wrong_tables_and_lengths():
    """Pages that the cache does not have, lengths below zero and past the table."""
    say("wrong tables")
    heads, kv, d, page, pages, width = 4, 2, 128, 16, 7, 20
    g = gen(6)
    held = mxq.KvCache(*(randn(g, pages, kv, page, d).to(DEV) for _ in range(2)))
    big, least = (1 << 31) - 1, -(1 << 31)
    table = torch.tensor([[least, big, -1, pages, 3] * 4, [big] * width, [pages - 1] * width, [0] * width], dtype=I32, device=DEV)
    q = randn(g, 4, heads, d)
    buf = torch.full((12, heads, d), 4.0, dtype=BF16, device=DEV)
    mxq.attention_paged(q.to(DEV), held, table, ints([320, 100, big, least]), out=buf[4:8])
    assert (buf[:4] == 4).all() and (buf[8:] == 4).all()
    assert not buf[5].any() and not buf[7].any()
    k, v = (t[3].transpose(0, 1).cpu().repeat(4, 1, 1) for t in held[:2])  # page 3, four times
    attention_check(buf[4:5], q[:1], k, v, [(1, len(k))], -1, -1, 0, d ** -0.5, "page 3")
    k, v = (t[pages - 1].transpose(0, 1).cpu().repeat(width, 1, 1) for t in held[:2])
    attention_check(buf[6:7], q[2:3], k, v, [(1, len(k))], -1, -1, 0, d ** -0.5, "last page")


# ------------------------------------------------------- rotary and plan ----

@pytest.mark.parametrize("fmt", [mxq.KV_BF16, mxq.KV_MXFP8])
def test_rotary_wrong_slots(fmt):
    """Slots at the ends of int32 and of the cache; a cache between guard pages."""
    say("wrong slots", fmt)
    kv, d, page, pages = 2, 128, 16, 3
    wide = mxq.kv_cache(pages + 2, kv, page, d, fmt)
    for t in wide:
        if t is not None:
            t.fill_(5)
    held = mxq.KvCache(*(None if t is None else t[1:1 + pages] for t in wide))
    big, least = (1 << 31) - 1, -(1 << 31)
    slots = [big, least, pages * page, -1, pages * page - 1, 0, big - 15, -page]
    x = randn(gen(7), len(slots), 3 * kv * d)
    _, k = mxq.rotary_qkv(x.to(DEV), kv, kv, d, cache=held, slots=ints(slots))
    for t in wide:
        if t is not None:
            assert (t[0] == 5).all() and (t[-1] == 5).all()
    written = (held.k.transpose(1, 2).reshape(pages * page, -1) != 5).any(1)
    assert torch.nonzero(written)[:, 0].tolist() == [0, pages * page - 1]
    if fmt == mxq.KV_BF16:
        assert torch.equal(held.k[0, :, 0], k[5]) and torch.equal(held.k[-1, :, -1], k[4])


@pytest.mark.parametrize("m, heads, kv, d, norm", [(1, 3, 1, 64, 2), (70001, 1, 0, 64, 2), (70001, 0, 1, 64, 0), (5, 1, 1, 128, 1)])
def test_rotary_few_heads(m, heads, kv, d, norm):
    """A workgroup of mostly idle threads, and many rows to each."""
    say("few heads", m, heads, kv, d, norm)
    x, freqs, axis, pos, weights = rotary_case(m, heads, kv, d, 8, 1, norm, m)
    pos = (torch.arange(m) * 3 - 50)[None].to(I32)
    w = [None if n == 0 or t is None else t.to(DEV) for n, t in zip((heads, kv), weights)]
    q, k = mxq.rotary_qkv(x.to(DEV), heads, kv, d, pos.to(DEV), freqs.to(DEV), axis.to(DEV), norm=norm, q_weight=w[0], k_weight=w[1])
    some = sorted(set(range(0, m, max(1, m // 50))) | set(range(max(0, m - 40), m)))
    want = rotary_want(x[some], heads, kv, d, freqs, axis, pos[:, some], weights, norm, False)
    for got, expect in zip((q, k), want):
        if got is not None:
            rotary_within(got[some], expect, "few heads")


def test_page_plan_wrong_lengths():
    """Lengths at the end of int32, whose sums wrap: the table's neighbours stay, and the next plan is right."""
    say("wrong lengths")
    big, least = (1 << 31) - 1, -(1 << 31)
    buf = torch.full((30, 5), 8, dtype=I32, device=DEV)
    for cached, added in (([big, big, 5], [big, big, big]), ([least, 0, big], [big, 1, least]), ([0, 0, 0], [big, big, 7])):
        buf.fill_(8)
        plan = mxq.page_plan(ints(cached), ints(added), buf[10:13], ints([1, 2, 3, 4]), 16, 40)
        torch.cuda.synchronize()
        assert (buf[:10] == 8).all() and (buf[13:] == 8).all() and len(plan.slots) == 40
    table = torch.full((1, 3), -1, dtype=I32, device=DEV)
    plan = mxq.page_plan(ints([0]), ints([20]), table, ints([6, 2]), 16, 20)
    assert plan.slots.tolist() == [96 + i for i in range(16)] + [32 + i for i in range(4)] and table.tolist() == [[6, 2, -1]]
