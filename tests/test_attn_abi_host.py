"""The C ABI and binding of the attention half on the host: include/mxq_attention.h and the library agree, and bad calls are
refused before any HIP call (no GPU needed)."""

import ctypes
import os
import re

import pytest
import torch

import mx_bit_quantized_amd as mxq
from conftest import ROOT
from mx_bit_quantized_amd import attn
from test_block_abi_host import FakeCuda, fake

HEADER = os.path.join(ROOT, "include", "mxq_attention.h")
P = 0x10000          # 16-byte aligned, never dereferenced
ODD = 0x10008        # 8-byte aligned only
OFF = 0x10002        # 2-byte aligned only
INF, NAN = float("inf"), float("nan")
i32 = torch.int32


def text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_library_exports_every_declared_symbol():
    names = set(re.findall(r"\b(mxq_[a-z0-9_]+)\s*\(", text()))
    assert names == set(attn._SIGS)
    for name in names:
        assert hasattr(mxq.lib(), name), name


@pytest.mark.parametrize("name, cls, size", [("mxq_kv_cache", attn.KvCacheArgs, 4 * 8 + 2 * 8 + 3 * 4 + 4),
                                             ("mxq_rotary_args", attn.RotaryArgs, 9 * 8 + 5 * 8 + 7 * 4 + 4),
                                             ("mxq_attention_args", attn.AttentionArgs, 6 * 8 + 10 * 8 + 3 * 4 + 4),
                                             ("mxq_paged_args", attn.PagedArgs, 4 * 8 + 6 * 8 + 4 + 4)])
def test_structs_match_the_header(name, cls, size):
    body = re.search(rf"typedef struct {name} \{{(.*?)\}}", text(), flags=re.S).group(1)
    declared = []
    for stmt in body.split(";"):
        stmt = re.sub(r"\b(const|void|float|double|int64_t|int32_t)\b|\*", " ", stmt)
        declared += [n.strip() for n in stmt.split(",") if n.strip()]
    assert declared == [n for n, _ in cls._fields_]
    assert ctypes.sizeof(cls) == size


def test_constants_match_the_header():
    for c, v in (("KV_BF16", 0), ("KV_MXFP8", 1), ("ROTARY_NORM_NONE", 0), ("ROTARY_NORM_ROW", 1), ("ROTARY_NORM_HEAD", 2)):
        assert re.search(rf"\bMXQ_{c} = {v}\b", text()) and getattr(mxq, c) == v
    assert re.search(rf"define MXQ_MAX_REQUESTS {mxq.MAX_REQUESTS}\b", text())


def plan(**change):
    a = dict(cached=P, added=P, table=P, free=P, requests=3, width=4, n_free=5, page=16, tokens=9, slots=P, positions=P, starts=P,
             lengths=P, taken=P)
    a.update(change)
    return attn._lib().mxq_page_plan(*a.values(), None)


@pytest.mark.parametrize("want, change", [(mxq.ERR_SHAPE, c) for c in (
    {"page": 0}, {"page": 8}, {"page": 24}, {"page": 2048}, {"requests": -1}, {"requests": mxq.MAX_REQUESTS + 1}, {"width": 0},
    {"width": 1 << 30}, {"n_free": -1}, {"n_free": 1 << 31}, {"tokens": -1}, {"tokens": 1 << 30})]
    + [(mxq.ERR_NULL, {n: None}) for n in ("cached", "added", "table", "free", "slots", "positions", "starts", "lengths", "taken")]
    + [(mxq.ERR_ALIGN, {n: OFF}) for n in ("cached", "added", "table", "free", "slots", "positions", "starts", "lengths", "taken")])
def test_page_plan_refuses(want, change):
    assert plan(**change) == want


def struct(cls, base, change):
    s = cls()
    for n, v in {**base, **change}.items():
        setattr(s, n, v)
    return s


CACHE = dict(k=P, v=P, pages=6, page_size=16, kv_heads=2, head_dim=64, format=0)
FP8 = dict(k_scales=P, v_scales=P, format=1)


def rotary(cache=None, **change):
    base = dict(qkv=P, positions=P, freqs=P, axis=P, q_weight=P, k_weight=P, q=P, k=P, M=5, ldx=512, ldq=256, ldk=128, ld_pos=5,
                heads=4, kv_heads=2, head_dim=64, axes=3, pairs=32, interleaved=1, norm=mxq.ROTARY_NORM_HEAD, eps=1e-6)
    if cache is not None:
        base["slots"] = P
        cache = ctypes.byref(struct(attn.KvCacheArgs, CACHE, cache))
    return attn._lib().mxq_rotary_qkv(ctypes.byref(struct(attn.RotaryArgs, base, change)), cache, None)


@pytest.mark.parametrize("want, change", [
    (mxq.ERR_MODE, {"norm": 3}), (mxq.ERR_MODE, {"norm": -1}), (mxq.ERR_MODE, {"eps": 0.0}), (mxq.ERR_MODE, {"eps": NAN}),
    (mxq.ERR_MODE, {"eps": INF}), (mxq.ERR_MODE, {"norm": 0}), (mxq.ERR_MODE, {"interleaved": 2}),
    (mxq.ERR_MODE, {"heads": 0, "ldx": 512}), (mxq.ERR_MODE, {"kv_heads": 0}),
    (mxq.ERR_SHAPE, {"head_dim": 96}), (mxq.ERR_SHAPE, {"head_dim": 32}), (mxq.ERR_SHAPE, {"heads": -1}),
    (mxq.ERR_SHAPE, {"heads": 0, "kv_heads": 0}), (mxq.ERR_SHAPE, {"heads": 2000}), (mxq.ERR_SHAPE, {"M": -1}),
    (mxq.ERR_SHAPE, {"heads": 1023, "ldx": 1 << 17}), (mxq.ERR_SHAPE, {"M": 1 << 30}), (mxq.ERR_SHAPE, {"ldx": 504}),
    (mxq.ERR_SHAPE, {"ldq": 128}), (mxq.ERR_SHAPE, {"ldk": 64}), (mxq.ERR_SHAPE, {"pairs": 12}), (mxq.ERR_SHAPE, {"pairs": 40}),
    (mxq.ERR_SHAPE, {"pairs": -8}), (mxq.ERR_SHAPE, {"axes": 0}), (mxq.ERR_SHAPE, {"ld_pos": 4}),
    (mxq.ERR_NULL, {"qkv": None}), (mxq.ERR_NULL, {"q": None}), (mxq.ERR_NULL, {"k": None}), (mxq.ERR_NULL, {"positions": None}),
    (mxq.ERR_NULL, {"freqs": None}), (mxq.ERR_NULL, {"slots": P}),
    (mxq.ERR_ALIGN, {"ldx": 516}), (mxq.ERR_ALIGN, {"ldq": 260}), (mxq.ERR_ALIGN, {"ldk": 132}), (mxq.ERR_ALIGN, {"freqs": 0x10004}),
] + [(mxq.ERR_ALIGN, {n: ODD}) for n in ("qkv", "q_weight", "k_weight", "q", "k")]
    + [(mxq.ERR_ALIGN, {n: OFF}) for n in ("positions", "axis")])
def test_rotary_refuses(want, change):
    assert rotary(**change) == want


@pytest.mark.parametrize("want, cache", [
    (mxq.ERR_MODE, {"format": 2}), (mxq.ERR_MODE, {"k_scales": P}), (mxq.ERR_SHAPE, {"head_dim": 128}), (mxq.ERR_SHAPE, {"kv_heads": 3}),
    (mxq.ERR_SHAPE, {"page_size": 8}), (mxq.ERR_SHAPE, {"page_size": 48}), (mxq.ERR_SHAPE, {"page_size": 2048}),
    (mxq.ERR_SHAPE, {"pages": 0}), (mxq.ERR_SHAPE, {"pages": 1 << 27}), (mxq.ERR_NULL, {"k": None}), (mxq.ERR_NULL, {"v": None}),
    (mxq.ERR_NULL, {"format": 1}), (mxq.ERR_NULL, {"format": 1, "k_scales": P}), (mxq.ERR_ALIGN, {"k": ODD}), (mxq.ERR_ALIGN, {"v": ODD}),
    (mxq.ERR_ALIGN, {**FP8, "k_scales": ODD}), (mxq.ERR_ALIGN, {**FP8, "v_scales": ODD})])
def test_rotary_refuses_caches(want, cache):
    assert rotary(cache=cache) == want
    assert rotary(cache=CACHE, slots=None) == mxq.ERR_NULL
    assert rotary(cache=CACHE, slots=OFF) == mxq.ERR_ALIGN


def test_rotary_empty():
    assert rotary(M=0, qkv=None, q=None, k=None, positions=None, freqs=None, axis=None) == mxq.OK
    assert attn._lib().mxq_rotary_qkv(None, None, None) == mxq.ERR_NULL


ATT = dict(q=P, k=P, v=P, starts_q=P, starts_k=P, out=P, sequences=2, Mq=5, Mk=9, ldq=256, ldk=128, ldv=128, ldo=256, left=-1, right=0,
           sinks=0, heads=4, kv_heads=2, head_dim=64, scale=0.125)


def attention(ws=(P, 1 << 40), **change):
    return attn._lib().mxq_attention(ctypes.byref(struct(attn.AttentionArgs, ATT, change)), *ws, None)


@pytest.mark.parametrize("want, change", [
    (mxq.ERR_MODE, {"scale": 0.0}), (mxq.ERR_MODE, {"scale": -1.0}), (mxq.ERR_MODE, {"scale": INF}), (mxq.ERR_MODE, {"scale": NAN}),
    (mxq.ERR_SHAPE, {"head_dim": 80}), (mxq.ERR_SHAPE, {"heads": 5}), (mxq.ERR_SHAPE, {"heads": 0}), (mxq.ERR_SHAPE, {"kv_heads": 0}),
    (mxq.ERR_SHAPE, {"heads": 2048}), (mxq.ERR_SHAPE, {"Mq": -1}), (mxq.ERR_SHAPE, {"Mk": -1}), (mxq.ERR_SHAPE, {"Mq": 1 << 30}),
    (mxq.ERR_SHAPE, {"Mk": 1 << 30}), (mxq.ERR_SHAPE, {"sequences": -1}), (mxq.ERR_SHAPE, {"sequences": 2, "starts_q": None}),
    (mxq.ERR_SHAPE, {"sequences": 2, "starts_k": None}), (mxq.ERR_SHAPE, {"sinks": -1}), (mxq.ERR_SHAPE, {"ldq": 128}),
    (mxq.ERR_SHAPE, {"ldk": 64}), (mxq.ERR_SHAPE, {"ldv": 64}), (mxq.ERR_SHAPE, {"ldo": 248}), (mxq.ERR_SHAPE, {"ldq": (1 << 24) + 8}),
    (mxq.ERR_SHAPE, {"Mq": (1 << 30) - 1, "heads": 1024, "kv_heads": 1024, "ldq": 1 << 16, "ldo": 1 << 16, "ldk": 1 << 16,
                     "ldv": 1 << 16}),
    (mxq.ERR_NULL, {"sequences": 1, "starts_q": None}), (mxq.ERR_NULL, {"sequences": 1, "starts_k": None}),
    (mxq.ERR_ALIGN, {"ldq": 260}), (mxq.ERR_ALIGN, {"ldk": 132}), (mxq.ERR_ALIGN, {"ldv": 132}), (mxq.ERR_ALIGN, {"ldo": 260}),
] + [(mxq.ERR_NULL, {n: None}) for n in ("q", "k", "v", "out")] + [(mxq.ERR_ALIGN, {n: ODD}) for n in ("q", "k", "v", "out")]
    + [(mxq.ERR_ALIGN, {n: OFF}) for n in ("starts_q", "starts_k")])
def test_attention_refuses(want, change):
    assert attention(**change) == want


def size_of(name, cls, base, change, *more):
    n = ctypes.c_size_t(77)
    st = getattr(attn._lib(), name)(ctypes.byref(struct(cls, base, change)), *more, ctypes.byref(n))
    return st, n.value


def test_attention_workspace():
    few = dict(Mq=3, Mk=1 << 20, sequences=1, starts_q=None, starts_k=None)
    st, need = size_of("mxq_attention_workspace_bytes", attn.AttentionArgs, ATT, few)
    assert st == mxq.OK and need > 0
    assert attention(ws=(None, need), **few) == mxq.ERR_WORKSPACE
    assert attention(ws=(P, need - 1), **few) == mxq.ERR_WORKSPACE
    assert attention(ws=(ODD, need), **few) == mxq.ERR_ALIGN
    many = dict(Mq=1 << 20, Mk=1 << 20, sequences=1, starts_q=None, starts_k=None)
    assert size_of("mxq_attention_workspace_bytes", attn.AttentionArgs, ATT, many) == (mxq.OK, 0)
    assert size_of("mxq_attention_workspace_bytes", attn.AttentionArgs, ATT, {"head_dim": 32}) == (mxq.ERR_SHAPE, 77)
    assert attn._lib().mxq_attention_workspace_bytes(None, ctypes.byref(ctypes.c_size_t())) == mxq.ERR_NULL
    assert attn._lib().mxq_attention(None, None, 0, None) == mxq.ERR_NULL


def test_attention_empty():
    none = dict(q=None, k=None, v=None, out=None, starts_q=None, starts_k=None)
    assert attention(ws=(None, 0), **none, sequences=1, Mq=0) == mxq.OK
    assert attention(ws=(None, 0), q=None, k=None, v=None, out=None, sequences=0) == mxq.OK


PAGED = dict(q=P, block_table=P, lengths=P, out=P, sequences=3, width=4, ldq=256, ldo=256, left=-1, sinks=0, heads=4, scale=0.125)


def paged(cache=(), ws=(P, 1 << 40), **change):
    c = ctypes.byref(struct(attn.KvCacheArgs, CACHE, dict(cache)))
    return attn._lib().mxq_attention_paged(ctypes.byref(struct(attn.PagedArgs, PAGED, change)), c, *ws, None)


@pytest.mark.parametrize("want, change", [
    (mxq.ERR_MODE, {"scale": 0.0}), (mxq.ERR_MODE, {"scale": NAN}), (mxq.ERR_SHAPE, {"heads": 3}), (mxq.ERR_SHAPE, {"heads": 0}),
    (mxq.ERR_SHAPE, {"sequences": -1}), (mxq.ERR_SHAPE, {"sequences": mxq.MAX_REQUESTS + 1}), (mxq.ERR_SHAPE, {"width": 0}),
    (mxq.ERR_SHAPE, {"sequences": 4096, "width": 1 << 18}), (mxq.ERR_SHAPE, {"sinks": -1}), (mxq.ERR_SHAPE, {"ldq": 248}),
    (mxq.ERR_SHAPE, {"ldo": 248}), (mxq.ERR_ALIGN, {"ldq": 260}), (mxq.ERR_ALIGN, {"ldo": 260}),
] + [(mxq.ERR_NULL, {n: None}) for n in ("q", "block_table", "lengths", "out")]
    + [(mxq.ERR_ALIGN, {n: ODD}) for n in ("q", "out")] + [(mxq.ERR_ALIGN, {n: OFF}) for n in ("block_table", "lengths")])
def test_paged_refuses(want, change):
    assert paged(**change) == want


@pytest.mark.parametrize("want, cache", [
    (mxq.ERR_MODE, {"format": 3}), (mxq.ERR_MODE, {"v_scales": P}), (mxq.ERR_SHAPE, {"head_dim": 96}), (mxq.ERR_SHAPE, {"kv_heads": 0}),
    (mxq.ERR_SHAPE, {"page_size": 4}), (mxq.ERR_SHAPE, {"pages": -1}), (mxq.ERR_NULL, {"k": None}), (mxq.ERR_NULL, {"format": 1})])
def test_paged_refuses_caches(want, cache):
    assert paged(cache=cache) == want


def test_paged_workspace_and_empty():
    c = ctypes.byref(struct(attn.KvCacheArgs, CACHE, {}))
    st, need = size_of("mxq_attention_paged_workspace_bytes", attn.PagedArgs, PAGED, {}, c)
    assert st == mxq.OK and need > 0
    assert paged(ws=(None, need)) == mxq.ERR_WORKSPACE and paged(ws=(P, need - 1)) == mxq.ERR_WORKSPACE
    assert paged(ws=(ODD, need)) == mxq.ERR_ALIGN
    assert paged(ws=(None, 0), sequences=0, q=None, out=None, block_table=None, lengths=None) == mxq.OK
    assert attn._lib().mxq_attention_paged(None, c, None, 0, None) == mxq.ERR_NULL


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    n = torch.zeros(4, dtype=i32)
    cache = mxq.KvCache(*(torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16) for _ in range(2)))
    for call in (lambda: mxq.attention(x, x, x), lambda: mxq.attention_paged(x, cache, n.view(4, 1), n),
                 lambda: mxq.rotary_qkv(x.view(4, 256), 2, 1, 64), lambda: mxq.page_plan(n, n, n.view(4, 1), n, 16, 4)):
        with pytest.raises(TypeError):
            call()


def test_binding_refuses_shapes_and_devices():
    q, k = fake(6, 4, 64), fake(9, 2, 64)
    starts = fake(3, dtype=i32)
    with pytest.raises(ValueError, match="k is on cuda:1"):
        mxq.attention(q, fake(9, 2, 64, device="cuda:1"), k)
    with pytest.raises(ValueError, match="v must have shape"):
        mxq.attention(q, k, fake(8, 2, 64))
    with pytest.raises(ValueError, match="k must have shape"):
        mxq.attention(q, fake(9, 2, 128), k)
    with pytest.raises(TypeError, match="q must have dtype"):
        mxq.attention(fake(6, 4, 64, dtype=torch.float16), k, k)
    with pytest.raises(ValueError, match="belong together"):
        mxq.attention(q, k, k, starts_q=starts)
    with pytest.raises(ValueError, match="starts_k must have shape"):
        mxq.attention(q, k, k, starts, fake(4, dtype=i32))
    with pytest.raises(TypeError, match="starts_k must have dtype"):
        mxq.attention(q, k, k, starts, fake(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="window counts"):
        mxq.attention(q, k, k, window=(-2, 0))
    with pytest.raises(ValueError, match="sinks must not"):
        mxq.attention(q, k, k, sinks=-1)
    with pytest.raises(ValueError, match="heads side by side"):
        mxq.attention(FakeCuda(torch.zeros(6, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), k, k)
    cache = mxq.KvCache(fake(3, 2, 16, 64), fake(3, 2, 16, 64))
    u8 = torch.uint8
    with pytest.raises(ValueError, match="heads of 64"):
        mxq.attention_paged(q, mxq.KvCache(fake(3, 2, 16, 128), fake(3, 2, 16, 128)), fake(6, 1, dtype=i32), fake(6, dtype=i32))
    with pytest.raises(ValueError, match="block_table must be"):
        mxq.attention_paged(q, cache, fake(5, 1, dtype=i32), fake(6, dtype=i32))
    with pytest.raises(ValueError, match="lengths must have shape"):
        mxq.attention_paged(q, cache, fake(6, 1, dtype=i32), fake(5, dtype=i32))
    with pytest.raises(TypeError, match="cache.k must have dtype"):
        mxq.attention_paged(q, mxq.KvCache(cache.k, cache.v, fake(3, 2, 16, 2, dtype=u8), fake(3, 2, 16, 2, dtype=u8)),
                            fake(6, 1, dtype=i32), fake(6, dtype=i32))
    with pytest.raises(ValueError, match="scales of its keys"):
        mxq.attention_paged(q, mxq.KvCache(cache.k, cache.v, fake(3, 2, 16, 2, dtype=u8)), fake(6, 1, dtype=i32), fake(6, dtype=i32))
    qkv, freqs, pos = fake(6, 512), fake(32, dtype=torch.float64), fake(6, dtype=i32)
    with pytest.raises(ValueError, match="columns"):
        mxq.rotary_qkv(qkv, 4, 1, 64)
    with pytest.raises(ValueError, match="needs positions"):
        mxq.rotary_qkv(qkv, 4, 2, 64, freqs=freqs)
    with pytest.raises(ValueError, match="belong to a rotation"):
        mxq.rotary_qkv(qkv, 4, 2, 64, positions=pos)
    with pytest.raises(ValueError, match="axis must have shape"):
        mxq.rotary_qkv(qkv, 4, 2, 64, pos, freqs, fake(31, dtype=i32))
    with pytest.raises(ValueError, match="q_weight must have shape"):
        mxq.rotary_qkv(qkv, 4, 2, 64, pos, freqs, norm=mxq.ROTARY_NORM_ROW, q_weight=fake(64))
    with pytest.raises(ValueError, match="cache and slots"):
        mxq.rotary_qkv(qkv, 4, 2, 64, pos, freqs, cache=cache)
    with pytest.raises(ValueError, match="output of a call with write_k"):
        mxq.rotary_qkv(qkv, 4, 2, 64, pos, freqs, k=k, write_k=False)
    n = fake(3, dtype=i32)
    with pytest.raises(ValueError, match="added must have shape"):
        mxq.page_plan(n, fake(2, dtype=i32), fake(3, 4, dtype=i32), n, 16, 5)
    with pytest.raises(ValueError, match="block_table must be"):
        mxq.page_plan(n, n, fake(2, 4, dtype=i32), n, 16, 5)
    with pytest.raises(ValueError, match="tokens must not"):
        mxq.page_plan(n, n, fake(3, 4, dtype=i32), n, 16, -5)


def test_frequencies():
    f, a = mxq.rotary_frequencies([22, 21, 21], 10000.0, device="cpu")
    assert f.dtype == torch.float64 and a.dtype == i32 and f.shape == a.shape == (64,)
    assert a.tolist() == [0] * 22 + [1] * 21 + [2] * 21
    assert f[0] == 1 and f[22] == 1 and f[11].item() == pytest.approx(10000.0 ** -0.5) and f[63].item() == pytest.approx(10000.0 ** (-20 / 21))
    f, a = mxq.rotary_frequencies(64, 1e6, device="cpu")
    assert f[32].item() == pytest.approx(1e-3) and not a.any()
