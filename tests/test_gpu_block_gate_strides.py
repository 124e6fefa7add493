"""mxq_gemm_residual with gates that are slices of a wider table, on both kernels and both ways the pipelined one reads a gate (one
group per tile: from the ring; several: row by row from memory), and the strides that it leaves to the split-K kernel.

A gate's stride changes no arithmetic, so the result equals that of the same gate packed densely, bit for bit, on the kernel that
the call is to run; the dense result is held to float64 in the same test."""

import pytest
import torch

import mx_bit_quantized_amd as mxq
from test_gpu_block import BF, DEV, KERNELS, U, bf16, block_kernel, gen, product, quantized, randn, rows_of, say, within

pytestmark = pytest.mark.gpu

F32, B16 = torch.float32, torch.bfloat16
CASES = [
    # m, n, k, type, rows per group, columns of the table before the slice and after it
    (300, 520, 640, F32, 100, 8, 0),    # tiles of several groups
    (300, 520, 640, B16, 7, 8, 56),
    (515, 776, 1280, F32, 1, 0, 16),    # a vector per row
    (515, 264, 640, B16, 256, 24, 8),   # one group per tile, not the first
    (700, 264, 672, F32, 512, 8, 8),
    (300, 520, 640, F32, None, 16, 8),  # one vector for all rows
    (33, 264, 512, B16, 3, 8, 8),
    (3, 264, 512, F32, 2, 0, 8),
]


def run(case, mode, dense):
    m, n, k, kind, rpg, before, after = case
    g = gen(m + n + k)
    a, w, A, W = quantized(mode, g, m, n, k)
    residual, bias = bf16(randn(g, m, n, scale=2.0)), bf16(randn(g, n, scale=0.5))
    table = randn(g, 1 if rpg is None else -(-m // rpg), before + n + after, scale=0.6).to(kind).to(DEV)
    gate = table[:, before:before + n]
    call = lambda t: mxq.gemm_residual(mode, *a, *w, residual.to(DEV), bias=bias.to(DEV), gate=t, rows_per_group=rpg)
    return call(gate.contiguous() if dense else gate), (A, W, residual, bias, gate.cpu())


def check(case, mode, got, operands):
    m, n, k, kind, rpg, *_ = case
    A, W, residual, bias, gate = operands
    v, err = product(A, W)
    v = v + bias.double()
    f = rows_of(gate, m, rpg or m)
    err = f.abs() * (err + 2 * U * v.abs())
    want = residual.double() + f * v
    within(got, want, err + BF * (want.abs() + err) + 2 * U * (residual.double().abs() + (f * v).abs()), "y")


@pytest.mark.parametrize("mode, waves, kernel", [k for k in KERNELS if k[1] == 4])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:3])))
def test_gate_as_a_slice_of_a_table(case, mode, waves, kernel):
    m, n, k, *_ = case
    say("gate slice", case, mode, kernel)
    with block_kernel(kernel):
        assert mxq.block_kernel_name(mode, m, n, k).startswith(kernel + "_")
        dense, operands = run(case, mode, True)
        sliced, _ = run(case, mode, False)
    check(case, mode, dense, operands)
    assert torch.equal(sliced, dense)


@pytest.mark.parametrize("mode", [mxq.W4A4, mxq.W4A8])
@pytest.mark.parametrize("case", [(300, 520, 640, F32, 100, 0, 4), (300, 520, 640, B16, 7, 8, 1), (515, 264, 640, B16, 256, 0, 2),
                                  (3, 33, 96, F32, 2, 4, 1), (40, 261, 512, B16, 3, 8, 0)], ids=lambda c: "x".join(map(str, c[:3])))
def test_strides_that_are_no_multiple_of_8(case, mode):
    """The split-K kernel's, also where the other one is asked for."""
    say("gate stride", case, mode)
    with block_kernel("tokens"):
        dense, operands = run(case, mode, True)
    check(case, mode, dense, operands)
    with block_kernel("pipe"):
        sliced, _ = run(case, mode, False)
    assert torch.equal(sliced, dense)
