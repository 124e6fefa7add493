"""The attention half's operators as a program uses them: together between the block's quantized products, over large buffers,
captured into graphs, on another stream, and under MXQ_CHECK_FINITE."""

import numpy as np
import pytest
import torch

import mx_bit_quantized_amd as mxq
import oracle
from test_gpu_attn import (BF, BF16, DEV, I32, attention_check, gen, host, ints, paged_check, randn, rotary_want, rotary_within, say,
                           within)
from test_gpu_check_finite import guard

pytestmark = pytest.mark.gpu

HEADS, KV, D, K, PAGE = 8, 2, 64, 512, 16
WIDTH = (HEADS + 2 * KV) * D


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    mxq.lib()
    yield
    torch.cuda.synchronize()


class Block:
    """The attention half of a block with quantized projections, and its cache."""

    def __init__(self, mode, fmt, pages, seed=1):
        g = gen(seed)
        self.mode = mode
        self.norm_weight = randn(g, K, scale=0.1).add_(1).to(DEV)
        self.w_qkv = mxq.quantize_weight_mxfp4(randn(g, WIDTH, K, scale=0.05).to(DEV))
        self.w_out = mxq.quantize_weight_mxfp4(randn(g, K, HEADS * D, scale=0.05).to(DEV))
        self.q_weight, self.k_weight = (randn(g, D, scale=0.1).add_(1.5).to(DEV) for _ in range(2))
        self.freqs, self.axis = mxq.rotary_frequencies(D // 2, 1e6)
        self.cache = mxq.kv_cache(pages, KV, PAGE, D, fmt)

    def projected(self, x):
        codes, scales, _ = mxq.norm_quantize(self.mode, x, weight=self.norm_weight)
        return mxq.gemm(self.mode, codes, scales, *self.w_qkv)

    def rotated(self, qkv, plan, **more):
        return mxq.rotary_qkv(qkv, HEADS, KV, D, plan.positions, self.freqs, norm=mxq.ROTARY_NORM_HEAD, q_weight=self.q_weight,
                              k_weight=self.k_weight, cache=self.cache, slots=plan.slots, **more)

    def output(self, o, x):
        return mxq.gemm_residual(self.mode, *mxq.quantize_act(self.mode, o.view(-1, HEADS * D)), *self.w_out, x)

    def prefill(self, x, plan, window=-1, sinks=0):
        """Tokens of several requests, nothing of them cached before: in place in the projection's rows."""
        qkv = self.projected(x)
        m = x.shape[0]
        q = qkv[:, :HEADS * D].view(m, HEADS, D)
        k = qkv[:, HEADS * D:(HEADS + KV) * D].view(m, KV, D)
        v = qkv[:, (HEADS + KV) * D:].view(m, KV, D)
        self.rotated(qkv, plan, q=q, k=k)
        o = mxq.attention(q, k, v, plan.starts, plan.starts, window=(window, 0), sinks=sinks)
        return o, self.output(o, x)

    def decode(self, x, plan, table, window=-1, sinks=0):
        """One new token per request."""
        q, _ = self.rotated(self.projected(x), plan, write_k=False)
        o = mxq.attention_paged(q, self.cache, table, plan.lengths, window=window, sinks=sinks)
        return o, self.output(o, x)


@pytest.mark.parametrize("mode", [mxq.W4A4, mxq.W4A8])
@pytest.mark.parametrize("fmt, window, sinks", [(mxq.KV_BF16, -1, 0), (mxq.KV_BF16, 30, 2), (mxq.KV_MXFP8, -1, 0)])
def test_block_half_prefill_then_decode(mode, fmt, window, sinks):
    """Prompts, then tokens one by one: the paged attention gives what attention gives on the whole sequences."""
    say("block", mode, fmt, window, sinks)
    prompts, steps = [37, 1, 100, 64], 3
    block = Block(mode, fmt, pages=60)
    b, g = len(prompts), gen(2)
    table = torch.full((b, 12), -1, dtype=I32, device=DEV)
    free = torch.randperm(60, generator=g).to(I32).to(DEV)
    m = sum(prompts)
    x = randn(g, m + 5, K).to(DEV)
    plan = mxq.page_plan(ints([0] * b), ints(prompts), table, free, PAGE, m + 5)
    assert plan.taken.tolist() == [sum(-(-n // PAGE) for n in prompts), 0]
    out, y = block.prefill(x, plan, window, sinks)
    # every row belongs to a sequence or is padding: the prompts' rows against the definition
    qkv = block.projected(x)
    angle_pos = plan.positions[None].cpu()
    want = rotary_want(qkv.cpu(), HEADS, KV, D, block.freqs.cpu(), block.axis.cpu(), angle_pos, [block.q_weight, block.k_weight], 2, False)
    q, k = mxq.rotary_qkv(qkv, HEADS, KV, D, plan.positions, block.freqs, norm=mxq.ROTARY_NORM_HEAD, q_weight=block.q_weight,
                          k_weight=block.k_weight)
    rotary_within(q, want[0], "q")
    v = qkv[:, (HEADS + KV) * D:].view(-1, KV, D)
    attention_check(out, q, k, v, [(n, n) for n in prompts], window, 0, sinks, D ** -0.5, "prefill")
    assert torch.equal(y[:m], block.output(out, x)[:m])
    history = [[t[s:s + n] for t in (k, v)] for s, n in zip(np.cumsum([0] + prompts[:-1]), prompts)]
    used, lengths = int(plan.taken[0]), list(prompts)
    for step in range(steps):
        x = randn(g, b, K).to(DEV)
        plan = mxq.page_plan(ints(lengths), ints([1] * b), table, free[used:], PAGE, b)
        used += int(plan.taken[0])
        lengths = [n + 1 for n in lengths]
        assert plan.lengths.tolist() == lengths and int(plan.taken[1]) == 0
        out, y = block.decode(x, plan, table, window, sinks)
        qkv = block.projected(x)
        q, k = block.rotated(qkv, plan)
        v = qkv[:, (HEADS + KV) * D:].view(-1, KV, D)
        rows = []
        for r in range(b):
            history[r] = [torch.cat([old, new[r:r + 1]]) for old, new in zip(history[r], (k, v))]
            held = history[r]
            if fmt == mxq.KV_MXFP8:
                held = [torch.from_numpy(oracle.mxfp8_dequantize(*oracle.mxfp8_quantize(host(t)))).to(BF16) for t in held]
            rows.append(held)
        paged_check(out, q, rows, lengths, window, sinks, D ** -0.5, f"decode {step}")
        starts_k = ints(np.cumsum([0] + lengths).tolist())
        whole = mxq.attention(q, torch.cat([r[0].to(DEV) for r in rows]), torch.cat([r[1].to(DEV) for r in rows]), ints(list(range(b + 1))),
                              starts_k, window=(window, 0), sinks=sinks)
        # each is off the definition by at most a bf16 half-step of the weights and one of the output, both below 2^-8 of the
        # largest value, and the fp32 sums by less than a tenth of that
        most = max(r[1].abs().max().item() for r in rows)
        assert (out.double() - whole.double()).abs().max().item() <= 2 * 2.2 * BF * most
        assert torch.equal(y, block.output(out, x))


def test_decode_step_captured_and_replayed():
    """A decoding step in a graph whose lengths, tables and tokens change between replays."""
    lengths, b = [40, 1, 90], 3
    block = Block(mxq.W4A8, mxq.KV_MXFP8, pages=40)
    for t in (block.cache.k, block.cache.v):
        t.random_(0, 0x78)
    for t in (block.cache.k_scales, block.cache.v_scales):
        t.random_(118, 121)
    table = torch.arange(b * 12, device=DEV, dtype=I32).view(b, 12)
    cached, added, free = ints(lengths), ints([1] * b), ints([37, 38, 39])
    x = randn(gen(7), b, K).to(DEV)

    def step():
        plan = mxq.page_plan(cached, added, table, free, PAGE, b)
        return block.decode(x, plan, table, 50, 2) + (plan.lengths, plan.slots)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        cached.copy_(ints([[40, 1, 90], [15, 16, 17], [0, 100, 33], [159, 0, 7]][i]))
        x.copy_(randn(gen(20 + i), b, K).to(DEV))
        state = [t.clone() for t in block.cache] + [table.clone()]
        eager = [t.clone() for t in step()]
        after = [t.clone() for t in block.cache] + [table.clone()]
        for t, was in zip((*block.cache, table), state):
            t.copy_(was)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(captured, eager):
            assert torch.equal(got, want), i
        for t, want in zip((*block.cache, table), after):
            assert torch.equal(t, want), i


@pytest.mark.parametrize("lens, window", [([(5, 3000)], -1), ([(70, 70), (200, 333)], 40)])
def test_attention_captured_and_replayed(lens, window):
    """Joined parts and ragged sequences whose starts change between replays."""
    g, heads, kv, d = gen(3), 4, 2, 128
    mq, mk = sum(n for n, _ in lens), sum(n for _, n in lens)
    q, k, v = randn(g, mq, heads, d).to(DEV), randn(g, mk, kv, d).to(DEV), randn(g, mk, kv, d).to(DEV)
    starts = [ints(np.concatenate([[0], np.cumsum([n[i] for n in lens])]).tolist()) for i in range(2)]
    out = torch.zeros(mq, heads, d, dtype=BF16, device=DEV)
    mxq.attention(q, k, v, *starts, window=(window, 0), out=out)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mxq.attention(q, k, v, *starts, window=(window, 0), out=out)
    for i in range(3):
        starts[0][0] = min(i, 4)  # the first rows belong to no sequence
        q.copy_(randn(gen(30 + i), mq, heads, d).to(DEV))
        out.fill_(3)
        eager = torch.full_like(out, 3)
        mxq.attention(q, k, v, *starts, window=(window, 0), out=eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and (out[:min(i, 4)] == 3).all()


def test_two_graphs_and_an_eager_call_together():
    """Calls on three streams at once, each with its own workspace."""
    g, heads, kv, d = gen(4), 10, 2, 128
    held = mxq.KvCache(*(randn(g, 200, kv, 64, d).to(DEV) for _ in range(2)))
    table = torch.randperm(200, generator=g)[:150].view(3, 50).to(I32).to(DEV)
    cases = [(randn(gen(50 + i), 3, heads, d).to(DEV), ints([3000 - 900 * i, 17 + i, 3200])) for i in range(3)]
    want = [mxq.attention_paged(q, held, table, n) for q, n in cases]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q, n in cases[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(mxq.attention_paged(q, held, table, n))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        eager = mxq.attention_paged(*cases[2][:1], held, table, cases[2][1], stream=streams[2])
        torch.cuda.synchronize()
        for got, w in zip(outs + [eager], want):
            assert torch.equal(got, w), i


def test_another_stream():
    """Every call on a stream of its own, while the current one is busy elsewhere."""
    s = torch.cuda.Stream()
    g = gen(5)
    x, pos = randn(g, 50, WIDTH).to(DEV), torch.arange(50, dtype=I32, device=DEV)
    freqs, _ = mxq.rotary_frequencies(D // 2)
    q, k = mxq.rotary_qkv(x, HEADS, KV, D, pos, freqs)
    v = x[:, (HEADS + KV) * D:].view(50, KV, D)
    o = mxq.attention(q, k, v, window=(-1, 0))
    torch.cuda.synchronize()
    q2, k2 = mxq.rotary_qkv(x, HEADS, KV, D, pos, freqs, stream=s)
    o2 = mxq.attention(q2, k2, v, window=(-1, 0), stream=s)
    plan = mxq.page_plan(ints([3]), ints([4]), torch.zeros(1, 2, dtype=I32, device=DEV), ints([5]), 16, 6, stream=s)
    s.synchronize()
    assert torch.equal(o, o2) and plan.slots.tolist() == [3, 4, 5, 6, -1, -1]


# ------------------------------------------------------- large buffers ----

def test_cache_past_4_gib():
    """Pages at the end of a cache whose keys alone take 8 GiB."""
    kv, d, page = 2, 128, 64
    pages = (1 << 33) // (2 * kv * page * d)
    held = mxq.KvCache(*(torch.empty(pages, kv, page, d, dtype=BF16, device=DEV) for _ in range(2)))
    m, heads = 130, 4
    ids = [pages - 1, 3, pages // 2 + 1]
    slots = torch.tensor([ids[i // page] * page + i % page for i in range(m)], dtype=I32, device=DEV)
    x = randn(gen(6), m, (heads + 2 * kv) * d).to(DEV)
    q, k = mxq.rotary_qkv(x, heads, kv, d, cache=held, slots=slots)
    v = x[:, (heads + kv) * d:].view(m, kv, d)
    for i, p in enumerate(ids):
        n = min(page, m - i * page)
        assert torch.equal(held.k[p, :, :n], k[i * page:i * page + n].transpose(0, 1))
        assert torch.equal(held.v[p, :, :n], v[i * page:i * page + n].transpose(0, 1))
    out = mxq.attention_paged(q[-1:], held, ints([ids]), ints([m]))
    attention_check(out, q[-1:], k, v, [(1, m)], -1, 0, 0, d ** -0.5, "far pages")


def test_rows_past_4_gib():
    """Strided rows of q, k, v and out more than 4 GiB apart."""
    m, heads, kv, d, ld = 40000, 2, 1, 64, 1 << 16
    buf = torch.empty(m, ld, dtype=BF16, device=DEV)  # 4.9 GiB
    x = buf[:, :(heads + 2 * kv) * d]
    x.copy_(randn(gen(7), 100, x.shape[1]).to(DEV).repeat(400, 1))
    q, k, v = x[:, :heads * d].view(m, heads, d), x[:, heads * d:(heads + kv) * d].view(m, kv, d), x[:, (heads + kv) * d:].view(m, kv, d)
    out = buf[:, ld // 2:ld // 2 + heads * d].view(m, heads, d)
    starts = ints([0, m - 300, m])
    mxq.attention(q, k, v, starts, starts, window=(50, 0), out=out)
    attention_check(out[-300:], q[-300:], k[-300:], v[-300:], [(300, 300)], 50, 0, 0, d ** -0.5, "far rows")
    q2, k2 = mxq.rotary_qkv(x, heads, kv, d, torch.full((m,), 1, dtype=I32, device=DEV), mxq.rotary_frequencies(d // 2)[0], q=q, k=k)
    assert q2 is q
    assert torch.equal(q[-100:], q[:100]) and torch.equal(k[-100:], k[:100]) and torch.isfinite(q[-100:]).all()


# -------------------------------------------------------- MXQ_CHECK_FINITE ----

def test_check_finite():
    g, m, heads, kv, d = gen(8), 20, 4, 2, 64
    x = randn(g, m, (heads + 2 * kv) * d).to(DEV)
    bad = x.clone()
    bad[3, 7] = float("inf")
    w, nan_w = torch.ones(d, dtype=BF16, device=DEV), torch.full((d,), float("nan"), dtype=BF16, device=DEV)
    out = torch.full((m, heads, d), 5.0, dtype=BF16, device=DEV)

    def refused(call):
        with pytest.raises(mxq.MxqError) as e:
            call()
        assert e.value.status == mxq.ERR_NONFINITE

    with guard(True):
        q, k = mxq.rotary_qkv(x, heads, kv, d, norm=mxq.ROTARY_NORM_HEAD, q_weight=w, k_weight=w)
        refused(lambda: mxq.rotary_qkv(bad, heads, kv, d, q=out))
        refused(lambda: mxq.rotary_qkv(x, heads, kv, d, norm=mxq.ROTARY_NORM_HEAD, q_weight=w, k_weight=nan_w, q=out))
        assert (out == 5).all()
        v = x[:, (heads + kv) * d:].view(m, kv, d)
        mxq.attention(q, k, v)
        for i, t in enumerate((q, k, v)):
            args = [a.clone() for a in (q, k, v)]
            args[i][m - 1, 0, 0] = float("nan")
            refused(lambda: mxq.attention(*args, out=out))
            assert (out == 5).all()
            # rows behind the last sequence may hold anything
            mxq.attention(*args, ints([0, m - 1]), ints([0, m - 1]), out=out.clone())
        cache = mxq.kv_cache(3, kv, 16, d)
        cache.k[2], cache.v[2] = float("nan"), float("nan")  # (a free page)
        table, n = ints([[0, 1]]), ints([20])
        mxq.attention_paged(q[:1], cache, table, n)
        qb = q[:1].clone()
        qb[0, 1, 2] = float("inf")
        refused(lambda: mxq.attention_paged(qb, cache, table, n))
        refused(lambda: mxq.attention_paged(q[:1], cache, ints([[0, 2]]), n))  # the output
    with guard(False):
        mxq.attention_paged(q[:1], cache, ints([[0, 2]]), n)
        torch.cuda.synchronize()
