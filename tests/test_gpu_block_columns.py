"""Products of one row with more columns than a grid of 1024 threads per 32 of them holds (2^27)."""

import pytest
import torch

import mx_bit_quantized_amd as mxq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_one_row_of_2_to_27_columns():
    n, k, last = 2 ** 27 + 32, 32, 96
    print("[case] residual", 1, n, k, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    a = mxq.quantize_act(mxq.W4A4, torch.randn(1, k, generator=g, device=DEV).to(torch.bfloat16))
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.zeros(mxq.mx_scale_shape(n, k), dtype=torch.uint8, device=DEV)
    scales[..., 0] = 120
    residual = torch.randn(1, n, generator=g, device=DEV, dtype=torch.bfloat16)
    y = mxq.gemm_residual(mxq.W4A4, *a, codes, scales, residual)
    for at in (0, 2 ** 26 - 64, 2 ** 27 - 64, n - last):  # a panel's rows are contiguous: any range of them is a weight
        part = mxq.gemm_residual(mxq.W4A4, *a, codes[at:at + last], scales[:, at:at + last], residual[:, at:at + last].contiguous())
        assert torch.equal(y[:, at:at + last], part), at
    torch.cuda.synchronize()
