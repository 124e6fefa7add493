"""A layer norm of a row of one value is its bias, exactly, whatever the row's length.

The sum of K <= 32768 equal bf16 values is exact in fp32 in any order (8 + 15 bits), and so is its K-th part, so a row's mean is
the value itself and nothing is left of it after the subtraction. A mean that is off by one step is not harmless there: the
difference, squared, is compared with eps, and becomes +-1 for values of a few thousand."""

import sys

import pytest
import torch

import mx_bit_quantized_amd as mxq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
VALUES = [0.0, 1.0, -1.5, 7.0, 100.0, -333.0, 1000.0, 65280.0, 1e5, -3.1e9, 1e-3, 2.0 ** -120]
# one, two and four chunks a thread; lengths of odd factors 7, 13, 21, 41, 47 and powers of two
LENGTHS = [224, 416, 672, 1312, 1504, 3584, 7168, 5120, 8992, 14336, 28672, 32768]


def rows(k, repeat=1):
    return torch.tensor(VALUES * repeat).to(torch.bfloat16)[:, None].expand(-1, k).contiguous().to(DEV)


@pytest.mark.parametrize("k", LENGTHS)
@pytest.mark.parametrize("repeat", [1, 400])  # one row and several rows a workgroup
def test_layer_norm_of_constant_rows_is_the_bias(k, repeat):
    if repeat > 1 and k > 8192:
        pytest.skip("one row at a time in either case")
    print("[case] constant rows", k, repeat, flush=True)
    sys.stdout.flush()
    g = torch.Generator(device=DEV)
    g.manual_seed(k)
    x = rows(k, repeat)
    bias = torch.randn(k, generator=g, device=DEV).to(torch.bfloat16)
    weight = torch.randn(k, generator=g, device=DEV).to(torch.bfloat16)
    out, _, _ = mxq.norm_quantize(mxq.POLICY_BF16, x, norm=mxq.NORM_LAYER, weight=weight, bias=bias)
    assert torch.equal(out, bias.expand_as(out))


@pytest.mark.parametrize("k", LENGTHS)
def test_post_norm_of_constant_branches_adds_its_bias(k):
    print("[case] constant branches", k, flush=True)
    sys.stdout.flush()
    g = torch.Generator(device=DEV)
    g.manual_seed(k + 1)
    branch = rows(k)
    x = torch.randn(branch.shape, generator=g, device=DEV).to(torch.bfloat16)
    bias = torch.randn(k, generator=g, device=DEV).to(torch.bfloat16)
    _, _, h = mxq.norm_quantize(mxq.POLICY_BF16, x, branch=branch, post_norm=mxq.NORM_LAYER, post_bias=bias)
    assert torch.equal(h, (x.float() + bias.float()).to(torch.bfloat16))
