"""norm_quantize whose bf16 output is x or the branch itself: each thread reads its part of a row before it writes it, whatever the
number of rows in flight."""

import pytest
import torch

import mx_bit_quantized_amd as mxq
from test_gpu_block import norm_inputs, run_norm, say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("post", [mxq.NORM_NONE, mxq.NORM_LAYER])
@pytest.mark.parametrize("out", ["x", "branch"])
# one row a workgroup, its loads ahead; two rows at a time, cut at the groups; two and four chunks a thread
@pytest.mark.parametrize("m, k, rpg", [(5, 96, 2), (700, 5120, 100), (4200, 5120, 7), (700, 8224, 3), (300, 16416, 128)])
def test_output_over_an_input(post, out, m, k, rpg):
    say("norm output over", out, m, k, post)
    case = (m, k, mxq.NORM_RMS, post, True, True, True, rpg, torch.float32, True, True)
    t = norm_inputs(case, m + k)
    want, _, h = run_norm(mxq.POLICY_BF16, case, t)
    over = dict(t, **{out: t[out].to(DEV)})
    got, _, h2 = run_norm(mxq.POLICY_BF16, case, over, out=over[out])
    assert got.data_ptr() == over[out].data_ptr()
    assert torch.equal(got, want) and torch.equal(h2, h)
