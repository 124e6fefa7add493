"""GPU tests of the loops of the attention half's kernels over more than a step: rows of one workgroup of rotary_qkv one after the
other, long pieces of a cache in one workgroup of attention_paged, uneven batches. Tolerances: those of test_gpu_attn.py."""

import numpy as np
import pytest
import torch

import mx_bit_quantized_amd as mxq
import oracle
from test_gpu_attn import BF16, DEV, I32, attention_check, gen, host, ints, randn, rotary_case, rotary_want, rotary_within, say

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- rotary ----
# A workgroup per step while there are at most 256 (1024 / its threads) steps of one or two rows; with more rows each workgroup
# takes several steps. Every row has a position and values of its own.

STEPS = [  # m, heads, kv, d, axes, norm, interleaved, cache, in place
    (1501, 40, 40, 128, 3, 1, True, None, False),       # row norm, a row a step, 6 steps
    (2563, 40, 40, 128, 3, 1, True, None, True),        # two rows a step, 6 steps, an odd end
    (2563, 40, 40, 128, 1, 1, False, mxq.KV_BF16, False),
    (601, 128, 128, 128, 3, 1, True, None, False),      # two units a thread, 3 steps
    (601, 128, 128, 128, 1, 1, False, mxq.KV_MXFP8, False),
    (601, 170, 170, 128, 3, 1, False, None, True),      # four units a thread
    (1037, 170, 170, 128, 1, 1, True, mxq.KV_BF16, False),
    (3001, 40, 8, 128, 1, 2, False, mxq.KV_BF16, False),    # norm per head, two rows a step
    (3001, 40, 8, 128, 1, 2, False, mxq.KV_MXFP8, True),
    (1999, 64, 64, 64, 3, 2, True, mxq.KV_MXFP8, False),    # a row a step
    (20011, 12, 4, 64, 3, 2, True, None, False),
]


@pytest.mark.parametrize("m, heads, kv, d, axes, norm, interleaved, cache, in_place", STEPS)
def test_rotary_steps(m, heads, kv, d, axes, norm, interleaved, cache, in_place):
    say("rotary steps", m, heads, kv, d, axes, norm, interleaved, cache, in_place)
    x, freqs, axis, _, weights = rotary_case(m, heads, kv, d, d // 2, axes, norm, m + heads)
    pos = torch.stack([torch.randperm(m, generator=gen(a + m)) * 97 + a for a in range(axes)]).to(I32)
    row_scale = torch.exp2(torch.randint(-6, 7, (m, 1), generator=gen(3 * m)).float())  # norms that differ from row to row
    x = (x.float() * row_scale).to(BF16)
    rows = x.to(DEV)
    page = 16
    pages = m // page + 2
    held = slots = None
    if cache is not None:
        held = mxq.kv_cache(pages, kv, page, d, cache)
        slots = torch.randperm(pages * page, generator=gen(m))[:m].to(I32)
        slots[::11] = -1
    out = {}
    if in_place:
        out = dict(q=rows[:, :heads * d].view(m, heads, d), k=rows[:, heads * d:(heads + kv) * d].view(m, kv, d))
    q, k = mxq.rotary_qkv(rows, heads, kv, d, pos.to(DEV), freqs.to(DEV), axis.to(DEV), interleaved=interleaved, norm=norm,
                          q_weight=weights[0].to(DEV), k_weight=weights[1].to(DEV), cache=held,
                          slots=None if slots is None else slots.to(DEV), **out)
    # a run of neighbouring rows at both ends and in the middle (whole workgroups), and some rows in between
    some = sorted({r for b in (0, m // 2, m - 14) for r in range(b, b + 14)} | set(range(5, m, max(1, m // 23))))
    want = rotary_want(x[some], heads, kv, d, freqs, axis, pos[:, some], weights, norm, interleaved)
    rotary_within(q[some], want[0], "q")
    rotary_within(k[some], want[1], "k")
    if in_place:
        assert torch.equal(rows[:, (heads + kv) * d:].cpu(), x[:, (heads + kv) * d:])
    if cache is None:
        return
    # every row of the cache: the dense k and v bit for bit, or their codes and scales
    kept = torch.nonzero(slots >= 0)[:, 0]
    at = slots[kept].long()
    v = x[:, (heads + kv) * d:].view(m, kv, d)
    for dense, codes, scales in ((k.cpu(), held.k, held.k_scales), (v, held.v, held.v_scales)):
        flat = codes.cpu().transpose(1, 2).reshape(pages * page, kv, d)
        if cache == mxq.KV_BF16:
            assert torch.equal(flat[at], dense[kept])
        else:
            flat_scales = scales.cpu().transpose(1, 2).reshape(pages * page, kv, d // 32)
            for part in torch.split(kept, 256):
                c, s = oracle.mxfp8_quantize(host(dense[part]))
                assert torch.equal(flat[slots[part].long()], torch.from_numpy(c))
                assert torch.equal(flat_scales[slots[part].long()], torch.from_numpy(s))
        free = torch.ones(pages * page, dtype=torch.bool)
        free[at] = False
        assert not flat[free].any()


# ----------------------------------------------------------------- paged ----
# A workgroup's piece is ceil(units / 512) units of 16 keys (heads of 64: / 768), units counted over sequences and key heads; a
# step of its four waves takes 8.

def long_paged(lengths, heads, kv, d, page, fmt, left, sinks, lost, steps, seed):
    g = gen(seed)
    counts = [-(-n // page) for n in lengths]
    seen_units = sum(-(-(n if left < 0 else min(n, left + 1)) // 16) for n in lengths) * kv
    assert seen_units / (512 if d == 128 else 768) > 8 * (steps - 1) + 1, "pieces of fewer steps"
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=g).tolist()
    table = np.full((len(lengths), max(counts) + 1), -1, np.int64)
    if fmt == mxq.KV_BF16:
        kc, vc = randn(g, pages, kv, page, d, scale=1.5), randn(g, pages, kv, page, d)
        held = mxq.KvCache(kc.to(DEV), vc.to(DEV))
    else:
        codes = [torch.randint(0, 127, (pages, kv, page, d), generator=g, dtype=torch.uint8) for _ in range(2)]
        codes = [c | (torch.randint(0, 2, c.shape, generator=g, dtype=torch.uint8) << 7) for c in codes]
        scales = [torch.randint(117, 120, (pages, kv, page, d // 32), generator=g, dtype=torch.uint8) for _ in range(2)]
        held = mxq.KvCache(*(t.to(DEV) for t in codes + scales))
    q = randn(g, len(lengths), heads, d, scale=1.5)
    checked = sorted({0, heads // kv - 1, heads - 1})
    rows = []
    for b, n in enumerate(lengths):
        ids = [order.pop() for _ in range(counts[b])]
        table[b, :len(ids)] = ids
        for col in lost.get(b, ()):
            table[b, col] = -1
        j = np.arange(n)
        seen = oracle.visible(n - 1, n, left, 0, sinks) & ~np.isin(j // page, lost.get(b, ()))
        keys = torch.from_numpy(j[seen])
        page_of, at = torch.tensor(ids)[keys // page], keys % page
        part = []
        for i in range(2):
            if fmt == mxq.KV_BF16:
                part.append((kc, vc)[i][page_of, :, at])
            else:
                part.append(torch.from_numpy(oracle.mxfp8_dequantize(codes[i][page_of, :, at].numpy(), scales[i][page_of, :, at].numpy()))
                            .to(BF16))
        rows.append(part)
    a = (q.to(DEV), held, torch.tensor(table, dtype=I32, device=DEV), ints(lengths))
    out = mxq.attention_paged(*a, window=left, sinks=sinks)
    for b, (k, v) in enumerate(rows):
        attention_check(out[b:b + 1], q[b:b + 1], k, v, [(1, len(k))], -1, -1, 0, d ** -0.5, f"sequence {b}", heads=checked)
    assert torch.equal(out, mxq.attention_paged(*a, window=left, sinks=sinks))


LONG = [  # lengths, heads, kv, d, page, left, sinks, lost columns of sequences, steps of a wave
    ([41507], 16, 8, 64, 16, -1, 0, {}, 3),
    ([28003], 8, 8, 128, 64, -1, 0, {}, 3),
    ([60001], 16, 8, 128, 16, -1, 0, {0: (7, 1900, 3750)}, 7),
    ([20011, 5, 33000, 1, 9001, 700], 8, 4, 128, 32, -1, 0, {}, 3),
    ([50021, 17, 40003, 3, 9001, 700], 8, 4, 64, 128, -1, 0, {2: (100, 101, 200)}, 3),
    ([30000, 50007, 26], 8, 8, 128, 16, 20000, 70, {0: (1000, 1500), 1: (2, 2500)}, 5),
    ([50000, 61009, 26, 30005], 8, 4, 64, 256, 33000, 300, {1: (150,)}, 4),
]


@pytest.mark.parametrize("lengths, heads, kv, d, page, left, sinks, lost, steps", LONG)
@pytest.mark.parametrize("fmt", [mxq.KV_BF16, mxq.KV_MXFP8])
def test_attention_paged_steps(lengths, heads, kv, d, page, left, sinks, lost, steps, fmt):
    say("paged steps", lengths, heads, kv, d, page, left, sinks, fmt)
    long_paged(lengths, heads, kv, d, page, fmt, left, sinks, lost, steps, sum(lengths) + d)


def test_attention_paged_maximum_late():
    """Keys whose scores grow along the cache, and keys far above all others in the last step of a piece: the running maximum
    moves at every step."""
    n, kv, d, page = 40003, 8, 128, 16
    say("paged, growing scores", n)
    g = gen(40)
    pages = -(-n // page)
    q = torch.ones(1, kv, d).to(BF16)
    grow = torch.linspace(0, 1.5, pages * page)
    k = (0.2 * torch.randn(pages * page, kv, d, generator=g) + grow[:, None, None])
    k[19999::2500] += 3.0
    k, v = k.to(BF16), randn(g, pages * page, kv, d)
    held = mxq.KvCache(*(t.view(pages, page, kv, d).transpose(1, 2).contiguous().to(DEV) for t in (k, v)))
    out = mxq.attention_paged(q.to(DEV), held, torch.arange(pages, dtype=I32, device=DEV)[None], ints([n]))
    attention_check(out, q, k[:n], v[:n], [(1, n)], -1, -1, 0, d ** -0.5, "growing", heads=[0, 7])


# ------------------------------------------------------------- attention ----

UNEVEN = [  # lens, heads, kv, d, left, right, sinks: one long axis among short ones, few rows each
    ([(1, 64)] * 32 + [(1, 30000)], 4, 2, 128, -1, 0, 0),
    ([(4, 100)] * 20 + [(4, 20011)] + [(4, 70)] * 11, 8, 8, 64, -1, 0, 0),
    ([(1, 9)] * 3 + [(2, 12000)], 4, 1, 128, -1, 0, 0),     # joined from parts, most of them empty for the short ones
    ([(3, 20), (5, 9000), (1, 1)], 4, 1, 64, 5000, 0, 70),
]


@pytest.mark.parametrize("lens, heads, kv, d, left, right, sinks", UNEVEN)
def test_attention_uneven_batches(lens, heads, kv, d, left, right, sinks):
    say("uneven", lens[:4], len(lens), heads, kv, d, left, right, sinks)
    g = gen(sum(n for _, n in lens))
    mq, mk = sum(n for n, _ in lens), sum(n for _, n in lens)
    q, k, v = randn(g, mq, heads, d, scale=1.5), randn(g, mk, kv, d, scale=1.5), randn(g, mk, kv, d)
    starts = [ints(np.concatenate([[0], np.cumsum([n[i] for n in lens])]).tolist()) for i in range(2)]
    out = mxq.attention(*(t.to(DEV) for t in (q, k, v)), *starts, window=(left, right), sinks=sinks)
    attention_check(out, q, k, v, lens, left, right, sinks, d ** -0.5, "uneven", heads=sorted({0, heads - 1}))
