"""MXQ_CHECK_FINITE on the operators around the linears: every bf16 and float32 vector of a call is scanned before anything is
written, and a value that overflows bf16 before it is quantized is reported, as it is in two steps (the bf16 values in memory,
then their quantizer)."""

import sys

import pytest
import torch

import mx_bit_quantized_amd as mxq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16
INF, NAN = float("inf"), float("nan")
BIG = float(torch.finfo(BF16).max)
M, K, RPG = 6, 256, 4  # two groups, the second of two rows
MODES = [mxq.W4A4, mxq.W4A8, mxq.POLICY_TRANSFORM_ON, mxq.POLICY_BF16]


@pytest.fixture(autouse=True)
def _guard(monkeypatch):
    monkeypatch.setenv("MXQ_CHECK_FINITE", "1")


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=BF16):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def norm_call(mode, mod_type, seed=1):
    """Arguments of a call with every vector, modulation as slices of one wider table, outputs filled with 7."""
    g = gen(seed)
    table = randn(g, 3, 4 * K, dtype=mod_type)
    kw = dict(x=randn(g, M, K), branch=randn(g, M, K), post_norm=mxq.NORM_RMS, norm=mxq.NORM_LAYER, rows_per_group=RPG,
              gate=table[:2, :K], scale=table[:2, K:2 * K], shift=table[:2, 2 * K:3 * K])
    for name in ("post_weight", "post_bias", "weight", "bias"):
        kw[name] = randn(g, K)
    kw.update(outputs(mode))
    return kw, table


def outputs(mode):
    kw = {"h": torch.full((M, K), 7.0, dtype=BF16, device=DEV)}
    if mode == mxq.POLICY_BF16:
        kw["out"] = torch.full((M, K), 7.0, dtype=BF16, device=DEV)
    else:
        kw["out"] = torch.full((M, K if mode == mxq.W4A8 else K // 2), 7, dtype=torch.uint8, device=DEV)
        kw["out_scales"] = torch.full((M,), 7.0, device=DEV) if mode == mxq.W4A8 else \
            torch.full(mxq.mx_scale_shape(M, K), 7, dtype=torch.uint8, device=DEV)
    if mode == mxq.POLICY_TRANSFORM_ON:
        kw["act_mult"] = torch.full((K,), 0.1, device=DEV)
    return kw


def refused(call):
    with pytest.raises(mxq.MxqError) as e:
        call()
    torch.cuda.synchronize()
    assert e.value.status == mxq.ERR_NONFINITE


VECTORS = [(mode, name) for mode in MODES for name in ("weight", "bias", "post_weight", "post_bias", "gate", "scale", "shift")]


@pytest.mark.parametrize("mode, name", VECTORS + [(mxq.POLICY_TRANSFORM_ON, "act_mult")])
@pytest.mark.parametrize("mod_type", [torch.float32, BF16])
def test_norm_refuses_a_bad_vector(mode, mod_type, name):
    say("norm vector", mode, mod_type, name)
    for bad in (INF, -INF, NAN):
        kw, _ = norm_call(mode, mod_type)
        kw[name][..., -1] = bad  # the last element, of every group
        refused(lambda: mxq.norm_quantize(mode, **kw))
        for out in ("h", "out", "out_scales"):
            assert out not in kw or (kw[out] == 7).all(), out


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("mod_type", [torch.float32, BF16])
def test_norm_accepts_bad_values_that_it_does_not_read(mode, mod_type):
    """Table columns between the vectors and a group that no row belongs to are no inputs."""
    kw, table = norm_call(mode, mod_type)
    table[:, 3 * K:] = NAN
    table[2] = NAN
    for name, c in (("gate", 0), ("scale", 1), ("shift", 2)):
        kw[name] = table[:, c * K:(c + 1) * K]  # three groups of 4 rows, 6 rows
    out, scales, h = mxq.norm_quantize(mode, **kw)
    assert torch.isfinite(h).all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("norm", [mxq.NORM_RMS, mxq.NORM_LAYER])
@pytest.mark.parametrize("write_h", [True, False])
def test_norm_reports_a_residual_stream_that_overflows(mode, norm, write_h):
    say("norm overflow of h", mode, norm, write_h)
    g = gen(2)
    x, branch = randn(g, M, K), randn(g, M, K)
    kw = {"act_mult": torch.full((K,), 0.1, device=DEV)} if mode == mxq.POLICY_TRANSFORM_ON else {}
    mxq.norm_quantize(mode, x, branch=branch, norm=norm, write_h=write_h, **kw)
    x[M - 1, K - 1] = branch[M - 1, K - 1] = BIG
    refused(lambda: mxq.norm_quantize(mode, x, branch=branch, norm=norm, write_h=write_h, **kw))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("m, k", [(1, 128), (5, 256), (300, 1152)])
def test_norm_reports_an_output_that_overflows(mode, m, k):
    """Finite inputs whose normalised value times the weight is past bf16."""
    say("norm overflow of n", mode, m, k)
    g = gen(3)
    x, weight = randn(g, m, k), torch.ones(k, dtype=BF16, device=DEV)
    kw = {"act_mult": torch.full((k,), 0.1, device=DEV)} if mode == mxq.POLICY_TRANSFORM_ON else {}
    x[m - 1, k - 1] = 10.0  # about nine times the row's norm
    mxq.norm_quantize(mode, x, weight=weight, **kw)
    weight[k - 1] = BIG
    refused(lambda: mxq.norm_quantize(mode, x, weight=weight, **kw))


@pytest.mark.parametrize("mode", [mxq.W4A4, mxq.W4A8])
def test_norm_of_the_largest_finite_values_is_accepted(mode):
    """n up to bf16's largest value: the largest scale that a finite block or row has."""
    x = torch.zeros(2, K, dtype=BF16, device=DEV)
    x[:, :K // 2] = 1.0
    x[:, K // 2:] = -1.0
    weight = torch.full((K,), BIG, dtype=BF16, device=DEV)
    n, _, _ = mxq.norm_quantize(mxq.POLICY_BF16, x, weight=weight, eps=1e-30)
    assert (n.abs().float() == BIG).all()
    codes, scales, _ = mxq.norm_quantize(mode, x, weight=weight, eps=1e-30)
    want, want_scales = mxq.quantize_act(mode, n)
    assert torch.equal(codes, want) and torch.equal(scales, want_scales)


def gated_operands(mode, m, h, k, seed=4, scale=1.0):
    g = gen(seed)
    a = mxq.quantize_act(mode, (scale * torch.randn(m, k, generator=g, device=DEV)).to(BF16))
    return a, mxq.quantize_weight_gated_mxfp4(randn(g, h, k), randn(g, h, k))


@pytest.mark.parametrize("m", [1, 300])
@pytest.mark.parametrize("mode, mxfp4_out", [(mxq.W4A4, True), (mxq.W4A4, False), (mxq.W4A8, False)])
@pytest.mark.parametrize("name", ["bias_gate", "bias_up"])
def test_gated_refuses_a_bad_bias(m, mode, mxfp4_out, name):
    say("gated bias", m, mode, mxfp4_out, name)
    h, k = 416, 512
    a, w = gated_operands(mode, m, h, k)
    for bad in (INF, -INF, NAN):
        bias = torch.zeros(h, dtype=BF16, device=DEV)
        bias[h - 1] = bad
        y = torch.full((m, h // 2), 7, dtype=torch.uint8, device=DEV) if mxfp4_out else torch.full((m, h), 7.0, dtype=BF16, device=DEV)
        ys = torch.full(mxq.mx_scale_shape(m, h), 7, dtype=torch.uint8, device=DEV) if mxfp4_out else None
        refused(lambda: mxq.gemm_gated(mode, *a, *w, mxq.GATED_SILU, y=y, y_scales=ys, **{name: bias}))
        assert (y == 7).all() and (ys is None or (ys == 7).all())


@pytest.mark.parametrize("m", [1, 300])
@pytest.mark.parametrize("mode, mxfp4_out", [(mxq.W4A4, True), (mxq.W4A4, False), (mxq.W4A8, False)])
def test_gated_reports_a_hidden_state_that_overflows(m, mode, mxfp4_out):
    """Finite operands whose act(g) u is past bf16 (products of about 1e30 each)."""
    say("gated overflow", m, mode, mxfp4_out)
    a, w = gated_operands(mode, m, 416, 512, scale=1e3)
    mxq.gemm_gated(mode, *a, *w, mxq.GATED_SILU, mxfp4_out=mxfp4_out)
    a, w = gated_operands(mode, m, 416, 512, scale=1e30)
    refused(lambda: mxq.gemm_gated(mode, *a, *w, mxq.GATED_SILU, mxfp4_out=mxfp4_out))


@pytest.mark.parametrize("m", [3, 300])
@pytest.mark.parametrize("mod_type", [torch.float32, BF16])
@pytest.mark.parametrize("n", [256, 261])
@pytest.mark.parametrize("name", ["bias", "gate"])
def test_residual_refuses_a_bad_vector(m, mod_type, n, name):
    """In place: a refused call leaves the residual stream as it was."""
    say("residual vector", m, mod_type, n, name)
    g = gen(5)
    k = 512
    a, w = mxq.quantize_act(mxq.W4A4, randn(g, m, k)), mxq.quantize_weight_mxfp4(randn(g, n, k))
    rpg = -(-m // 2)
    gate = randn(g, 2, n + 3, dtype=mod_type)[:, :n]
    bias = randn(g, n)
    y = torch.full((m, n), 7.0, dtype=BF16, device=DEV)
    for bad in (INF, NAN):
        vec = {"bias": bias.clone(), "gate": gate}
        vec[name][..., n - 1] = bad
        refused(lambda: mxq.gemm_residual(mxq.W4A4, *a, *w, y, rows_per_group=rpg, y=y, **vec))
        assert (y == 7).all()
        vec[name][..., n - 1] = 1.0
    assert torch.isfinite(mxq.gemm_residual(mxq.W4A4, *a, *w, y, bias=bias, gate=gate, rows_per_group=rpg)).all()
