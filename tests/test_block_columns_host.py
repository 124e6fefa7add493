"""The products refuse more columns than a grid of the split-K kernel holds, 2^32 threads of 512 to 32 columns (no GPU needed)."""

import mx_bit_quantized_amd as mxq
from test_block_abi_host import gated, residual

MOST = 2 ** 28 - 32


def test_columns_past_a_grid_are_refused():
    assert residual(N=MOST, gate=None, M=0) == mxq.OK
    assert residual(N=MOST + 1, gate=None, M=0) == mxq.ERR_SHAPE
    assert residual(N=MOST + 1, gate=None) == mxq.ERR_SHAPE
    assert gated(H=MOST, M=0) == mxq.OK
    assert gated(H=MOST + 32, M=0) == mxq.ERR_SHAPE
    assert gated(H=MOST + 32) == mxq.ERR_SHAPE
