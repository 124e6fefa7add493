"""GPU tests of the forms that the attention calls choose by size: workgroups of 256 rows, keys in parts, the largest batch, rows
far apart, windows past every position. Tolerances: those of test_gpu_attn.py."""

import numpy as np
import pytest
import torch

import mx_bit_quantized_amd as mxq
import oracle
from test_gpu_attn import BF, BF16, DEV, U, attention_check, gen, host, ints, paged_check, randn, say

pytestmark = pytest.mark.gpu


WIDE = [  # lens, heads, kv, left, right, sinks: long axes and rows for all CUs, heads of 128
    ([(1100, 6200)], 64, 8, -1, 0, 0),
    ([(1031, 6145)], 64, 64, -1, -1, 0),
    ([(700, 7000), (0, 13), (340, 12000)], 64, 16, 6200, 100, 3),
    ([(1, 6300), (1050, 6200), (3, 6000)], 64, 1, -1, 5, 0),
]


@pytest.mark.parametrize("lens, heads, kv, left, right, sinks", WIDE)
def test_attention_wide(lens, heads, kv, left, right, sinks):
    say("wide", lens, heads, kv, left, right, sinks)
    g, d = gen(heads + kv), 128
    mq, mk = sum(n for n, _ in lens) + 3, sum(n for _, n in lens)
    q, k, v = randn(g, mq, heads, d, scale=1.5), randn(g, mk, kv, d, scale=1.5), randn(g, mk, kv, d)
    starts = [ints(np.concatenate([[0], np.cumsum([n[i] for n in lens])]).tolist()) for i in range(2)]
    out = torch.full((mq, heads, d), 3.0, dtype=BF16, device=DEV)
    mxq.attention(q.to(DEV), k.to(DEV), v.to(DEV), *starts, window=(left, right), sinks=sinks, out=out)
    assert (out[mq - 3:] == 3).all()
    attention_check(out, q, k, v, lens, left, right, sinks, d ** -0.5, "wide", heads=(0, heads - 1))


def test_attention_wide_hidden_places_hold_anything():
    nq, nk, heads, kv, d, left, right = 1030, 6400, 64, 1, 128, 6200, 20
    g = gen(17)
    q, k, v = randn(g, nq, heads, d), randn(g, nk, kv, d), randn(g, nk, kv, d)
    first = nk - nq
    k[first + 70, 0, 1], k[2, 0, 0] = float("inf"), float("nan")
    v[nk - 30, 0, 3], v[nk - 31, 0, 4], v[first + 31, 0, 33] = float("nan"), float("inf"), -float("inf")
    out = host(mxq.attention(q.to(DEV), k.to(DEV), v.to(DEV), window=(left, right)))
    clean = 0
    for h in (0, 31, 63):
        with np.errstate(all="ignore"):
            o, mean, top = oracle.attention_rows(host(q)[:, h], host(k)[:, 0], host(v)[:, 0], first, left, right, 0, d ** -0.5)
        for i in range(nq):
            if np.isnan(o[i]).all():
                assert np.isnan(out[i, h]).all(), i
                continue
            fine = np.isfinite(o[i])
            clean += fine.sum()
            assert np.array_equal(np.isnan(o[i]), np.isnan(out[i, h])) and np.array_equal(o[i][~fine], out[i, h][~fine], equal_nan=True), i
            off = (2 * (2 * d + 8 + 4 * (nk // 64 + 2)) * U * top[i] + 2.0 ** -19 + BF) * mean[i][fine]
            assert (np.abs(out[i, h][fine] - o[i][fine]) <= BF * (np.abs(o[i][fine]) + off) + off).all(), i
    # every row sees the NaN key or the value of -inf; those past the NaN key whose score with the infinite one is -inf (half
    # of 197, for each head) have all but one to three columns finite
    assert clean > 20 * (d - 3)


PARTS = [  # nq, nk, heads, kv, d, left, right
    (1, 129, 8, 8, 128, -1, 0),       # two tiles and a key
    (2, 700, 8, 2, 64, -1, 0),
    (16, 8000, 10, 2, 128, -1, 0),
    (100, 4000, 40, 40, 128, -1, -1),
    (37, 30011, 8, 1, 64, -1, 0),
    (3, 20000, 4, 4, 128, 3000, 2),   # parts of a window
    (9, 5000, 1, 1, 64, 4999, 0),
]


@pytest.mark.parametrize("nq, nk, heads, kv, d, left, right", PARTS)
def test_attention_in_parts(nq, nk, heads, kv, d, left, right):
    say("parts", nq, nk, heads, kv, d, left, right)
    g = gen(nq + nk)
    q, k, v = randn(g, nq, heads, d, scale=1.5), randn(g, nk, kv, d, scale=1.5), randn(g, nk, kv, d)
    out = mxq.attention(q.to(DEV), k.to(DEV), v.to(DEV), window=(left, right))
    attention_check(out, q, k, v, [(nq, nk)], left, right, 0, d ** -0.5, "parts", heads=sorted({0, heads - 1}))


@pytest.mark.parametrize("d, nq", [(64, 70), (128, 33)])
def test_attention_rows_far_apart(d, nq):
    """Row strides of 2^24 elements, the most: 32 MiB from row to row."""
    say("far apart", d, nq)
    ld, heads, kv, nk = 1 << 24, 4, 2, 70
    g = gen(d)
    buf = torch.empty(max(nq, nk), ld, dtype=BF16, device=DEV)
    cut = [0, heads * d, (heads + kv) * d, (heads + 2 * kv) * d, (2 * heads + 2 * kv) * d]
    q, k, v, out = (buf[:n, cut[i]:cut[i + 1]].view(n, -1, d) for i, n in enumerate((nq, nk, nk, nq)))
    for t in (q, k, v):
        t.copy_(randn(g, *t.shape).to(DEV))
    mxq.attention(q, k, v, window=(-1, 0), out=out)
    attention_check(out, q, k, v, [(nq, nk)], -1, 0, 0, d ** -0.5, "far apart")


def test_attention_windows_past_every_position():
    g = gen(8)
    q, k, v = (randn(g, 200, 2, 64).to(DEV) for _ in range(3))
    for big in (199, 200, (1 << 63) - 1, 1 << 80):
        for wide, none in (((big, big), (-1, -1)), ((big, 0), (-1, 0))):
            assert torch.equal(mxq.attention(q, k, v, window=wide, sinks=big), mxq.attention(q, k, v, window=none)), big


@pytest.mark.parametrize("d, fmt", [(128, mxq.KV_BF16), (64, mxq.KV_MXFP8)])
def test_attention_paged_largest_batch(d, fmt):
    """As many sequences as a call takes, one page each or none, all at the same pages."""
    say("largest batch", d, fmt)
    n, heads, kv, page, pages = mxq.MAX_REQUESTS, 4, 2, 16, 5
    g = gen(d)
    x = randn(g, pages * page, 2 * kv * d)
    held = mxq.kv_cache(pages, kv, page, d, fmt, DEV)
    mxq.rotary_qkv(x.to(DEV), 0, kv, d, cache=held, slots=ints(list(range(pages * page))), write_k=False)
    k, v = (x[:, i * kv * d:(i + 1) * kv * d].view(-1, kv, d) for i in range(2))
    if fmt == mxq.KV_MXFP8:
        k, v = (torch.from_numpy(oracle.mxfp8_dequantize(*oracle.mxfp8_quantize(host(t)))).to(BF16) for t in (k, v))
    lengths = [(7 * b) % 17 for b in range(n)]
    table = torch.tensor([[b % pages] for b in range(n)], dtype=torch.int32, device=DEV)
    q = randn(g, n, heads, d)
    out = mxq.attention_paged(q.to(DEV), held, table, ints(lengths))
    assert not out[[b for b in range(n) if lengths[b] == 0]].any()
    for b in list(range(0, n, 97)) + [n - 1]:
        rows = [(t[(b % pages) * page:][:lengths[b]]) for t in (k, v)]
        paged_check(out[b:b + 1], q[b:b + 1], [rows], [lengths[b]], -1, 0, d ** -0.5, f"sequence {b} of the batch")
