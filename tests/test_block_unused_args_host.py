"""mxq_norm_quantize refuses operands that its mode does not read, as it refuses a post_weight without a post_norm (no GPU needed)."""

import pytest

import mx_bit_quantized_amd as mxq
from test_block_abi_host import P, norm

WIDE = dict(K=128, ldx=128, ldb=128, ldh=128, ld_mod=128)


@pytest.mark.parametrize("mode", [mxq.W4A4, mxq.W4A8, mxq.POLICY_BF16])
def test_factors_without_the_transform(mode):
    scales = None if mode == mxq.POLICY_BF16 else P
    assert norm(mode, act_mult=P, out_scales=scales, **WIDE) == mxq.ERR_MODE


def test_scales_of_a_bf16_output():
    assert norm(mxq.POLICY_BF16) == mxq.ERR_MODE


def test_an_empty_problem_is_no_error():
    assert norm(mxq.W4A4, M=0, act_mult=P) == mxq.OK
    assert norm(mxq.POLICY_BF16, M=0) == mxq.OK
