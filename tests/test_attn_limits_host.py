"""Host tests of what the attention calls take at the ends of their ranges (include/mxq_attention.h)."""

import ctypes

import pytest

import mx_bit_quantized_amd as mxq
from mx_bit_quantized_amd import attn
from test_attn_abi_host import ATT, CACHE, PAGED, attention, paged, size_of, struct

FEW = dict(Mq=3, Mk=1 << 20, sequences=1, starts_q=None, starts_k=None)


@pytest.mark.parametrize("scale", [2.0 ** 127, 3e38])
def test_scales_whose_log2_overflows(scale):
    assert attention(scale=scale) == mxq.ERR_MODE
    assert paged(scale=scale) == mxq.ERR_MODE


@pytest.mark.parametrize("left, right", [((1 << 63) - 1, (1 << 63) - 1), (1 << 62, 1 << 62), (0, (1 << 63) - 1), ((1 << 63) - 1, 0)])
def test_windows_past_every_position(left, right):
    none = size_of("mxq_attention_workspace_bytes", attn.AttentionArgs, ATT, dict(FEW, left=-1, right=-1))
    assert none[0] == mxq.OK and none[1] > 0
    assert size_of("mxq_attention_workspace_bytes", attn.AttentionArgs, ATT, dict(FEW, left=left, right=right, sinks=(1 << 63) - 1)) == none


def test_parts_go_by_the_keys_that_rows_see():
    seen = [size_of("mxq_attention_workspace_bytes", attn.AttentionArgs, ATT, dict(FEW, left=n, right=0))[1] for n in (100, 2000, 1 << 20)]
    assert seen[0] == 0 and 0 < seen[1] <= seen[2]
    rows = [size_of("mxq_attention_workspace_bytes", attn.AttentionArgs, ATT, dict(FEW, Mq=m))[1] for m in (1, 1000, 1 << 20)]
    assert rows[0] > 0 and rows[2] == 0


def test_binding_takes_windows_of_any_size():
    assert attn._window(1 << 70, -1, 1 << 64) == (1 << 62, -1, 1 << 62)
    for bad in ((-2, 0, 0), (0, -2, 0), (0, 0, -1)):
        with pytest.raises(ValueError):
            attn._window(*bad)


def test_largest_paged_batch_has_a_workspace():
    c = ctypes.byref(struct(attn.KvCacheArgs, CACHE, {}))
    small = size_of("mxq_attention_paged_workspace_bytes", attn.PagedArgs, PAGED, {}, c)
    large = size_of("mxq_attention_paged_workspace_bytes", attn.PagedArgs, PAGED, dict(sequences=mxq.MAX_REQUESTS), c)
    assert small[0] == large[0] == mxq.OK and small[1] < large[1] <= small[1] + 4 * mxq.MAX_REQUESTS
