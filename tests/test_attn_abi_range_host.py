"""Host tests of counts at the ends of the ranges of their types (include/mxq_attention.h): refused, without arithmetic that
overflows on the way (the sanitized run of these tests watches that)."""

import pytest

import mx_bit_quantized_amd as mxq
from test_attn_abi_host import attention, paged, plan, rotary

I32_MAX, I32_MIN, I64_MAX, I64_MIN = (1 << 31) - 1, -(1 << 31), (1 << 63) - 1, -(1 << 63)


# multiples of 8 whose double is past 2^31, and one whose double wraps to 0
@pytest.mark.parametrize("pairs", [1 << 30, (1 << 30) + 32, I32_MAX - 7, I32_MIN, I32_MIN + 32])
def test_rotary_refuses_pairs(pairs):
    assert rotary(pairs=pairs) == mxq.ERR_SHAPE
    assert rotary(pairs=pairs, interleaved=0) == mxq.ERR_SHAPE
    assert rotary(pairs=pairs, M=0) == mxq.ERR_SHAPE


@pytest.mark.parametrize("change", [{"heads": I32_MAX}, {"kv_heads": I32_MAX}, {"heads": I32_MAX, "kv_heads": I32_MAX},
                                    {"heads": I32_MIN}, {"heads": I32_MIN, "kv_heads": I32_MIN}, {"heads": 1, "kv_heads": I32_MAX},
                                    {"head_dim": I32_MAX}, {"head_dim": I32_MIN}, {"axes": I32_MIN}, {"M": I64_MAX}, {"M": I64_MIN},
                                    {"ldx": I64_MAX}, {"ldx": I64_MIN}, {"ldq": I64_MAX}, {"ldk": I64_MAX}, {"ld_pos": I64_MAX}])
def test_rotary_refuses_counts(change):
    assert rotary(**change) == mxq.ERR_SHAPE


@pytest.mark.parametrize("cache", [{"pages": I64_MAX}, {"pages": I64_MIN}, {"page_size": I64_MAX}, {"page_size": I64_MIN},
                                   {"kv_heads": I32_MAX}, {"kv_heads": I32_MIN}, {"head_dim": I32_MIN}])
def test_caches_refused(cache):
    assert rotary(cache=cache) == mxq.ERR_SHAPE
    assert paged(cache=cache) == mxq.ERR_SHAPE


@pytest.mark.parametrize("change", [{n: v} for n in ("sequences", "Mq", "Mk", "ldq", "ldk", "ldv", "ldo") for v in (I64_MAX, I64_MIN)]
                         + [{n: v} for n in ("heads", "kv_heads", "head_dim") for v in (I32_MAX, I32_MIN)] + [{"sinks": I64_MIN}])
def test_attention_refuses_counts(change):
    assert attention(**change) == mxq.ERR_SHAPE


@pytest.mark.parametrize("change", [{n: v} for n in ("sequences", "width", "ldq", "ldo") for v in (I64_MAX, I64_MIN)]
                         + [{"heads": I32_MAX}, {"heads": I32_MIN}, {"sinks": I64_MIN}])
def test_paged_refuses_counts(change):
    assert paged(**change) == mxq.ERR_SHAPE


@pytest.mark.parametrize("change", [{n: v} for n in ("page", "requests", "width", "n_free", "tokens") for v in (I64_MAX, I64_MIN)])
def test_page_plan_refuses_counts(change):
    assert plan(**change) == mxq.ERR_SHAPE


@pytest.mark.parametrize("norm", [mxq.ROTARY_NORM_ROW, mxq.ROTARY_NORM_HEAD])
@pytest.mark.parametrize("eps", [1e-40, 2.0 ** -127, 2.0 ** -149, -1e-6])
def test_rotary_refuses_subnormal_eps(eps, norm):
    assert rotary(eps=eps, norm=norm) == mxq.ERR_MODE
    assert rotary(eps=2.0 ** -126, norm=norm, M=0) == mxq.OK
    assert rotary(eps=eps, norm=mxq.ROTARY_NORM_NONE, q_weight=None, k_weight=None, M=0) == mxq.OK
