"""Which kernel the block operators' products take where MXQ_BLOCK_KERNEL asks for the pipelined one: the shapes that the GPU tests run
under that name do run it (no GPU needed)."""

import pytest

import mx_bit_quantized_amd as mxq
from test_gpu_block import GATED_CASES, RESIDUAL_CASES, block_kernel

STAGES = {mxq.W4A4: 4, mxq.W4A8: 3}  # panels of 128 elements that a tile needs


def pipelined(mode, n, k):
    """The pipelined kernel's shapes: n columns of the product, whole panels of K (and perhaps a ragged one)."""
    return n >= 256 and n % 8 == 0 and k // 128 >= STAGES[mode]


@pytest.mark.parametrize("mode, suffix", [(mxq.W4A4, "w4a4"), (mxq.W4A8, "w4a8")])
def test_the_pipelined_kernel_takes_its_shapes(mode, suffix):
    taken = 0
    for gated, cases in ((False, RESIDUAL_CASES), (True, GATED_CASES)):
        for m, n, k, *_ in cases:
            want = pipelined(mode, 2 * n if gated else n, k)
            with block_kernel("pipe"):
                assert mxq.block_kernel_name(mode, m, n, k, gated=gated) == ("pipe_" if want else "tokens_") + suffix, (m, n, k)
                if gated and mode == mxq.W4A4:
                    assert mxq.block_kernel_name(mode, m, n, k, gated=True, mxfp4_out=True).startswith("pipe_") == want
            with block_kernel("tokens"):
                assert mxq.block_kernel_name(mode, m, n, k, gated=gated) == "tokens_" + suffix
            taken += want
    assert taken >= 24


@pytest.mark.parametrize("k, mode, want", [(512, mxq.W4A4, True), (544, mxq.W4A4, True), (480, mxq.W4A4, False), (384, mxq.W4A4, False),
                                           (384, mxq.W4A8, True), (416, mxq.W4A8, True), (352, mxq.W4A8, False)])
def test_panels_that_a_tile_needs(k, mode, want):
    with block_kernel("pipe"):
        assert mxq.block_kernel_name(mode, 300, 256, k).startswith("pipe_") == want
        assert mxq.block_kernel_name(mode, 300, 128, k, gated=True).startswith("pipe_") == want
        assert mxq.block_kernel_name(mode, 300, 260, k).startswith("tokens_")
        assert mxq.block_kernel_name(mode, 300, 248, k).startswith("tokens_")
