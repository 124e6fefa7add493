"""Rows whose squares sum past fp32's range are no finite inputs of a norm: their output is NaN, not the finite bias that a reciprocal
root of infinity would leave, and MXQ_CHECK_FINITE reports it in every format. Rows just inside the range are normalised."""

import pytest
import torch

import mx_bit_quantized_amd as mxq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16
MODES = [mxq.W4A4, mxq.W4A8, mxq.POLICY_TRANSFORM_ON, mxq.POLICY_BF16]
SIZES = [(5, 256), (3, 8960), (2, 17024)]  # one, two and four chunks a thread


def factors(mode, k):
    return {"act_mult": torch.full((k,), 0.1, device=DEV)} if mode == mxq.POLICY_TRANSFORM_ON else {}


def stream(m, k, value):
    g = torch.Generator(device=DEV)
    g.manual_seed(k)
    x = torch.randn(m, k, generator=g, device=DEV).to(BF16)
    x[m - 1, 3] = value
    return x


@pytest.mark.parametrize("norm", [mxq.NORM_RMS, mxq.NORM_LAYER])
@pytest.mark.parametrize("m, k", SIZES)
def test_row_past_the_range_is_nan_and_the_others_stay(m, k, norm):
    print("[case] range", m, k, norm, flush=True)
    bias = torch.ones(k, dtype=BF16, device=DEV)
    want, _, _ = mxq.norm_quantize(mxq.POLICY_BF16, stream(m, k, 1.0), norm=norm, bias=bias)
    out, _, _ = mxq.norm_quantize(mxq.POLICY_BF16, stream(m, k, 2e19), norm=norm, bias=bias)
    assert torch.isnan(out[m - 1]).all()
    assert torch.equal(out[:m - 1], want[:m - 1])
    # 2^63: squared 2^126; the row is that value among zeros (the rest is below 2^-60 of it)
    out, _, _ = mxq.norm_quantize(mxq.POLICY_BF16, stream(m, k, 2.0 ** 63), norm=norm, bias=bias)
    x = torch.zeros(k, dtype=torch.float64)
    x[3] = 1.0
    if norm == mxq.NORM_LAYER:
        x = x - x.mean()
    n = x / x.square().mean().sqrt() + 1
    # half a bf16 step, and 32 fp32 half steps of the value and of the row's mean magnitude in units of its norm
    tol = 2.0 ** -8 * n.abs() + 2.0 ** -24 * (32 * (n - 1).abs() + 32 + 8)
    assert ((out[m - 1].cpu().double() - n).abs() <= tol).all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("m, k", SIZES)
@pytest.mark.parametrize("where", ["x", "branch"])
def test_guard_reports_a_row_past_the_range(monkeypatch, mode, m, k, where):
    print("[case] range guard", mode, m, k, where, flush=True)
    monkeypatch.setenv("MXQ_CHECK_FINITE", "1")
    t = {"x": stream(m, k, 1.0), "branch": stream(m, k, 1.0)}
    call = lambda: mxq.norm_quantize(mode, t["x"], branch=t["branch"], post_norm=mxq.NORM_RMS, write_h=False, **factors(mode, k))
    call()
    t[where][m - 1, 3] = 2e19
    with pytest.raises(mxq.MxqError) as e:
        call()
    assert e.value.status == mxq.ERR_NONFINITE
