"""The attention half's oracle against torch on the CPU and closed forms (no GPU needed)."""

import numpy as np
import pytest
import torch

import oracle


def test_mxfp8_round_trip_and_torch():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((40, 128)) * np.exp2(rng.integers(-20, 20, (40, 1)))).to(torch.bfloat16)
    codes, scales = oracle.mxfp8_quantize(x.double().numpy())
    back = oracle.mxfp8_dequantize(codes, scales)
    again, same = oracle.mxfp8_quantize(back)
    assert np.array_equal(oracle.mxfp8_dequantize(again, same), back)
    assert np.array_equal(torch.from_numpy(back).to(torch.bfloat16).double().numpy(), back)  # bf16 numbers
    b = x.float().view(40, 4, 32)
    e = torch.floor(torch.log2(b.abs().amax(-1))) - 8
    q = (b * torch.exp2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert np.array_equal(codes, q.view(torch.uint8).view(40, 128).numpy())
    assert np.array_equal(scales, (e + 127).to(torch.uint8).numpy())


def test_mxfp8_zero_and_saturation():
    x = np.zeros((1, 32))
    codes, scales = oracle.mxfp8_quantize(x)
    assert not codes.any() and not scales.any()
    x[0, 0], x[0, 1] = 1.9921875, -1.0  # amax / scale = 510: saturates at 448
    codes, scales = oracle.mxfp8_quantize(x)
    assert scales[0, 0] == 127 - 8 and codes[0, 0] == 0x7E
    assert oracle.mxfp8_dequantize(codes, scales)[0, 1] == -1.0


def test_rotation_keeps_norms_and_composes():
    rng = np.random.default_rng(2)
    x, a, b = rng.standard_normal((5, 64)), rng.uniform(-9, 9, (5, 16)), rng.uniform(-9, 9, (5, 16))
    for interleaved in (False, True):
        y = oracle.rotate(x, a, interleaved)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[:, 32:], x[:, 32:])
        assert np.allclose(oracle.rotate(y, b, interleaved), oracle.rotate(x, a + b, interleaved))
    z = oracle.rotate(x, a, True)[:, 0:32:2] + 1j * oracle.rotate(x, a, True)[:, 1:32:2]
    assert np.allclose(z, (x[:, 0:32:2] + 1j * x[:, 1:32:2]) * np.exp(1j * a))


@pytest.mark.parametrize("left, right, sinks", [(-1, -1, 0), (-1, 0, 0), (5, 0, 2), (3, 4, 0), (0, 0, 0)])
def test_attention_rows_against_torch(left, right, sinks):
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((7, 16)), rng.standard_normal((19, 16)), rng.standard_normal((19, 16))
    first = 12
    out, _, _ = oracle.attention_rows(q, k, v, first, left, right, sinks, 0.25)
    mask = torch.from_numpy(np.stack([oracle.visible(first + i, 19, left, right, sinks) for i in range(7)]))
    s = (torch.from_numpy(q) @ torch.from_numpy(k).T * 0.25).masked_fill(~mask, -np.inf)
    assert np.allclose(out, (torch.softmax(s, -1) @ torch.from_numpy(v)).numpy())
    # row by row: key j of query i
    for i in range(7):
        for j in range(19):
            p = first + i
            want = (right < 0 or j <= p + right) and (left < 0 or j >= p - left or j < sinks)
            assert mask[i, j] == want


def test_attention_rows_of_nothing():
    q, k, v = np.ones((3, 4)), np.full((2, 4), np.nan), np.full((2, 4), np.nan)
    out, _, _ = oracle.attention_rows(q, k, v, -3, -1, 0, 0, 1.0)  # every key lies in the future
    assert not out.any()
    assert oracle.attention_rows(q, k[:0], v[:0], 0, -1, -1, 0, 1.0)[0].shape == (3, 4)


def test_page_plan_by_hand():
    table = [[7, -1, -1], [3, 4, -1], [-1, -1, -1]]
    slots, positions, starts, lengths, taken, after = oracle.page_plan([3, 8, 0], [2, 5, 1], table, [9, 1, 2], 4, 10)
    assert positions == [3, 4, 8, 9, 10, 11, 12, 0, 0, 0]
    assert starts == [0, 2, 7, 8] and lengths == [5, 13, 1]
    assert after.tolist() == [[7, 9, -1], [3, 4, 1], [2, -1, -1]]
    # request 1's last token lies behind the table
    assert slots == [31, 36, 4, 5, 6, 7, -1, 8, -1, -1] and taken == [3, 1]
