"""GPU tests of the operators around the quantized linears (include/mxq_block.h).

Each result is compared with the operator's definition in float64 on the CPU, computed from the same stored operands
(the library's own codes, decoded; its own bf16 h). Tolerances, with u = 2^-24 (half an fp32 step) and 2^-8 (half a bf16
step) relative to the value:

* norm: the sum of squares (and the mean) passes at most 8 + 4 + 6 + 4 additions in depth, so it is off by less than 24 u of
  its terms' magnitudes; square root, division and the four products that follow add less than 8 u. A normalised value is
  thus off by 32 u of itself plus 32 u of the row's mean magnitude, in units of the row's norm.
* products: the fp32 sum of K exact products is off by at most one step, 2 u, per addition: 2 K u sum |a| |w|.
* activations: 1 / (1 + exp(-v)) is off by 4 u and the exponent's argument by 2 u |v|; both stay below 2^-15 for |v| < 100.
  Their slopes are below 1.2.
"""

import contextlib
import os
import sys

import numpy as np
import pytest
import torch

import mx_bit_quantized_amd as mxq
from gpu_util import assert_codes_equal, host_u8, w4a4_waves

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
DEV = "cuda:0"
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    mxq.lib()
    yield
    torch.cuda.synchronize()


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, scale=1.0, mean=0.0):
    return mean + scale * torch.randn(*shape, generator=g)


def bf16(t):
    return t.to(torch.bfloat16)


def activation(g, m, k):
    x = randn(g, m, k)
    x[:, torch.randperm(k, generator=g)[:max(1, k // 100)]] *= 10
    return bf16(x)


def decode_mxfp4(codes, scales, rows, k):
    """Library layout on the GPU -> float64 values on the CPU."""
    c, s = mxq.mxfp4_to_canonical(codes, scales, rows, k)
    c, s = c.cpu(), s.cpu()
    v = torch.stack((E2M1[(c & 15).long()], E2M1[(c >> 4).long()]), dim=2).view(rows, k)
    return v * torch.exp2(s.double() - 127).repeat_interleave(32, dim=1)


def decode_act(mode, codes, scales, m, k):
    if mode == mxq.W4A4:
        return decode_mxfp4(codes, scales, m, k)
    return codes.view(torch.float8_e4m3fn).float().cpu().double() * scales.cpu().double()[:, None]


def within(got, want, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = (got - want).abs() - tol
    assert over.max() <= 0, f"{what}: off by {float((got - want).abs().max())}, {int((over > 0).sum())} past tolerance, " \
                            f"worst at {np.unravel_index(int(over.argmax()), tuple(over.shape))}"


@contextlib.contextmanager
def block_kernel(name):
    """The products' kernel fixed to the split-K ("tokens") or the pipelined one ("pipe") where it takes the shape."""
    old = os.environ.get("MXQ_BLOCK_KERNEL")
    os.environ["MXQ_BLOCK_KERNEL"] = name
    try:
        yield
    finally:
        if old is None:
            os.environ.pop("MXQ_BLOCK_KERNEL", None)
        else:
            os.environ["MXQ_BLOCK_KERNEL"] = old


# mode, waves of the W4A4 pipelined kernel, kernel
KERNELS = [(mxq.W4A4, 4, "pipe"), (mxq.W4A4, 8, "pipe"), (mxq.W4A4, 4, "tokens"), (mxq.W4A8, 4, "pipe"), (mxq.W4A8, 4, "tokens")]


# ------------------------------------------------------------------- norm ----

def norm64(v, kind):
    """(normalised values, bound of their error per unit) of float64 rows."""
    mag = v.abs().mean(1, keepdim=True)
    if kind == mxq.NORM_LAYER:
        v = v - v.mean(1, keepdim=True)
    else:
        mag = torch.zeros_like(mag)
    r = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    return v * r, 32 * U * (v.abs() * r + mag * r)


def rows_of(t, m, rpg):
    t = t.double()
    if t.dim() == 1:
        return t.expand(m, -1)
    return t[torch.arange(m) // rpg]


NORM_CASES = [
    # m, k, norm, post_norm, branch, gate, modulated, rows_per_group, modulation type, weight, bias
    (1, 5120, mxq.NORM_RMS, 0, True, False, False, None, torch.float32, True, False),
    (1, 32, mxq.NORM_LAYER, 0, False, False, False, None, torch.float32, False, False),
    (3, 96, mxq.NORM_RMS, mxq.NORM_RMS, True, True, True, 2, torch.bfloat16, True, True),
    (5, 160, mxq.NORM_LAYER, mxq.NORM_LAYER, True, True, True, 1, torch.float32, True, True),
    (70, 1056, mxq.NORM_LAYER, 0, True, True, True, 17, torch.float32, False, False),
    (257, 512, mxq.NORM_RMS, mxq.NORM_LAYER, True, True, False, 100, torch.bfloat16, True, False),
    (33, 8192, mxq.NORM_LAYER, 0, True, True, True, 33, torch.float32, True, True),
    (9, 8224, mxq.NORM_RMS, mxq.NORM_RMS, True, True, True, 4, torch.bfloat16, True, True),
    (4, 16416, mxq.NORM_LAYER, mxq.NORM_LAYER, True, True, True, 3, torch.float32, True, True),
    (2, 32768, mxq.NORM_RMS, 0, True, False, True, None, torch.float32, True, False),
    (4099, 256, mxq.NORM_LAYER, 0, True, True, True, 1000, torch.float32, True, True),
    (9001, 224, mxq.NORM_RMS, mxq.NORM_RMS, True, True, True, 7, torch.bfloat16, True, True),
    (12289, 128, mxq.NORM_RMS, 0, True, False, True, 1, torch.float32, False, False),
]


def norm_inputs(case, seed):
    m, k, norm, post, branch, gate, mod, rpg, mod_type, weight, bias = case
    g = gen(seed)
    groups = None if rpg is None else -(-m // rpg)
    vec = (lambda mean, std: randn(g, k, scale=std, mean=mean).to(mod_type)) if groups is None else \
        (lambda mean, std: randn(g, groups, k, scale=std, mean=mean).to(mod_type))
    t = {"x": bf16(randn(g, m, k) + 0.5)}
    if branch:
        t["branch"] = bf16(randn(g, m, k, scale=2.0, mean=-0.25))
    if gate:
        t["gate"] = vec(0.4, 0.5)
    if mod:
        t["scale"], t["shift"] = vec(0.0, 0.3), vec(0.1, 0.3)
    if weight:
        t["weight"] = bf16(randn(g, k, scale=0.2, mean=1.0))
    if bias:
        t["bias"] = bf16(randn(g, k, scale=0.2))
    if post and weight:
        t["post_weight"] = bf16(randn(g, k, scale=0.2, mean=0.7))
    if post and bias:
        t["post_bias"] = bf16(randn(g, k, scale=0.2))
    return t


def run_norm(mode, case, t, **more):
    m, k, norm, post, *_ = case
    rpg = case[7]
    d = {n: v.to(DEV) for n, v in t.items()}
    return mxq.norm_quantize(mode, d.pop("x"), norm=norm, post_norm=post, rows_per_group=rpg, branch_scale=more.pop("branch_scale", 1.0),
                             **d, **more)


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: f"{c[0]}x{c[1]}")
def test_norm_matches_float64(case):
    m, k, norm, post, branch, gate, mod, rpg, *_ = case
    say("norm", case)
    t = norm_inputs(case, 11 + m + k)
    s = 0.75 if branch else 1.0
    out, scales, h = run_norm(mxq.POLICY_BF16, case, t, branch_scale=s)
    assert scales is None
    x = t["x"].double()
    if branch:
        b, err = t["branch"].double(), torch.zeros(m, k, dtype=torch.float64)
        if post:
            b, err = norm64(b, post)
        if "post_weight" in t:
            b, err = b * t["post_weight"].double(), err * t["post_weight"].double().abs()
        if "post_bias" in t:
            b = b + t["post_bias"].double()
        f = s * (rows_of(t["gate"], m, rpg) if gate else torch.ones(m, k, dtype=torch.float64))
        want = x + f * b
        within(h, want, BF * want.abs() + err * f.abs() + 8 * U * (x.abs() + (f * b).abs() + f.abs()), "h")
    else:
        assert h.data_ptr() != 0 and torch.equal(h.cpu(), t["x"])
    v, err = norm64(h.cpu().double(), norm)
    a = t["weight"].double() if "weight" in t else torch.ones(k, dtype=torch.float64)
    o = t["bias"].double() if "bias" in t else torch.zeros(k, dtype=torch.float64)
    a, o = a.expand(m, k), o.expand(m, k)
    if mod:
        sc, sh = rows_of(t["scale"], m, rpg), rows_of(t["shift"], m, rpg)
        a, o_mag, o = a * (1 + sc), (o * (1 + sc)).abs() + sh.abs(), o * (1 + sc) + sh
    else:
        o_mag = o.abs()
    want = v * a + o
    within(out, want, BF * want.abs() + err * a.abs() + 8 * U * ((v * a).abs() + o_mag), "n")


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: f"{c[0]}x{c[1]}")
def test_norm_codes_are_those_of_the_bf16_output(case):
    m, k = case[:2]
    say("norm codes", case)
    t = norm_inputs(case, 23 + m + k)
    n, _, h = run_norm(mxq.POLICY_BF16, case, t)
    for mode in (mxq.W4A4, mxq.W4A8):
        codes, scales, h2 = run_norm(mode, case, t)
        rc, rs = mxq.quantize_act(mode, n)
        assert torch.equal(h2, h)
        assert_codes_equal(host_u8(codes), host_u8(rc), f"codes {mode}")
        assert_codes_equal(host_u8(scales), host_u8(rs), f"scales {mode}")
    if k % 128 == 0:
        mult = randn(gen(5), k, scale=0.02, mean=0.1).to(DEV)
        codes, scales, _ = run_norm(mxq.POLICY_TRANSFORM_ON, case, t, act_mult=mult)
        rc, rs = mxq.quantize_mxfp4_hadamard(n, mult)
        assert_codes_equal(host_u8(codes), host_u8(rc), "transformed codes")
        assert_codes_equal(host_u8(scales), host_u8(rs), "transformed scales")


def test_norm_of_rows_of_zeros_and_of_one_value():
    k = 256
    x = torch.zeros(5, k, dtype=torch.bfloat16)
    x[1] = 3.0       # a layer norm of a constant row is its bias
    x[2, 7] = 1e-20  # far below eps
    x[3] = 1e15
    bias = bf16(randn(gen(3), k))
    for norm in (mxq.NORM_RMS, mxq.NORM_LAYER):
        out, _, _ = mxq.norm_quantize(mxq.POLICY_BF16, x.to(DEV), norm=norm, bias=bias.to(DEV))
        v, err = norm64(x.double(), norm)
        want = v + bias.double()
        within(out, want, BF * want.abs() + err + 8 * U * (v.abs() + 1), f"norm {norm}")
        for mode in (mxq.W4A4, mxq.W4A8):  # without a bias the rows of zeros stay zeros, codes and scales too
            codes, scales, _ = mxq.norm_quantize(mode, x.to(DEV), norm=norm)
            n, _, _ = mxq.norm_quantize(mxq.POLICY_BF16, x.to(DEV), norm=norm)
            rc, rs = mxq.quantize_act(mode, n)
            assert torch.equal(codes, rc) and torch.equal(scales, rs)


@pytest.mark.parametrize("alias", ["x", "branch"])
@pytest.mark.parametrize("m, k", [(3, 96), (4500, 512)])
def test_norm_in_place(alias, m, k):
    case = (m, k, mxq.NORM_RMS, mxq.NORM_RMS, True, True, False, 5, torch.float32, True, False)
    t = norm_inputs(case, 31)
    want = run_norm(mxq.POLICY_BF16, case, t)
    d = {n: v.to(DEV) for n, v in t.items()}
    got = mxq.norm_quantize(mxq.POLICY_BF16, d["x"], branch=d["branch"], gate=d["gate"], weight=d["weight"],
                            post_weight=d["post_weight"], post_norm=mxq.NORM_RMS, rows_per_group=5, h=d[alias])
    assert got[2].data_ptr() == d[alias].data_ptr()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    other = "branch" if alias == "x" else "x"
    assert torch.equal(d[other].cpu(), t[other])


@pytest.mark.parametrize("mode", [mxq.W4A4, mxq.W4A8, mxq.POLICY_BF16])
@pytest.mark.parametrize("m, k", [(2, 160), (4300, 160)])
def test_norm_strided_rows_and_nothing_written_around(mode, m, k):
    """Rows of wider buffers, modulation as slices of one table; what lies around the outputs keeps its values."""
    g = gen(41)
    xs, bs = bf16(randn(g, m, k + 64)).to(DEV), bf16(randn(g, m, k + 8)).to(DEV)
    table = randn(g, 3, 6 * k, scale=0.3).to(DEV)
    rpg = -(-m // 3)
    hs = torch.full((m + 2, k + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    kw = dict(gate=table[:, 2 * k:3 * k], scale=table[:, k:2 * k], shift=table[:, :k], rows_per_group=rpg)
    n_out = mxq.norm_quantize(mode, xs[:, 32:32 + k].contiguous(), branch=bs[:, :k].contiguous(), **{
        key: v.contiguous() if isinstance(v, torch.Tensor) else v for key, v in kw.items()})
    width = {mxq.W4A4: k // 2, mxq.W4A8: k, mxq.POLICY_BF16: k}[mode]
    dt = torch.bfloat16 if mode == mxq.POLICY_BF16 else torch.uint8
    guard = torch.full((m + 4, width), 3, dtype=dt, device=DEV)
    out = guard[2:m + 2]
    if out.data_ptr() % 16:
        pytest.skip("guard rows of this width are not aligned")
    scales = None
    got = mxq.norm_quantize(mode, xs[:, 32:32 + k], branch=bs[:, :k], h=hs[1:m + 1, 8:8 + k], out=out, out_scales=scales, **kw)
    assert torch.equal(got[0], n_out[0]) and torch.equal(got[2], n_out[2])
    if mode != mxq.POLICY_BF16:
        assert torch.equal(got[1], n_out[1])
    assert (guard[:2] == 3).all() and (guard[m + 2:] == 3).all()
    assert (hs[0] == 7).all() and (hs[m + 1] == 7).all() and (hs[:, :8] == 7).all() and (hs[:, 8 + k:] == 7).all()


# --------------------------------------------------------------- products ----

def quantized(mode, g, m, n, k, gated=False):
    """Operands on the GPU and their float64 values: ((a, a_scales), (w, w_scales), A, W or (Wg, Wu))."""
    a = mxq.quantize_act(mode, activation(g, m, k).to(DEV))
    if gated:
        wg, wu = bf16(randn(g, n, k, scale=0.05)), bf16(randn(g, n, k, scale=0.05))
        w = mxq.quantize_weight_gated_mxfp4(wg.to(DEV), wu.to(DEV))
        W = decode_mxfp4(*w, 2 * n, k).view(n // 32, 2, 32, k)
        W = (W[:, 0].reshape(n, k), W[:, 1].reshape(n, k))
    else:
        w = mxq.quantize_weight_mxfp4(bf16(randn(g, n, k, scale=0.05)).to(DEV))
        W = decode_mxfp4(*w, n, k)
    return a, w, decode_act(mode, *a, m, k), W


def product(A, W):
    """Float64 product and the bound of an fp32 sum's error."""
    return A @ W.T, 2 * A.shape[1] * U * (A.abs() @ W.abs().T)


def gelu64(v):
    return 0.5 * v * (1 + torch.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))


def act64(v, act):
    return v * torch.sigmoid(v) if act == mxq.GATED_SILU else gelu64(v)


RESIDUAL_CASES = [
    # m, n, k, bias, gelu, gate type, rows per group
    (1, 32, 32, False, False, None, None),
    (1, 5120, 640, False, False, None, None),
    (3, 33, 96, True, False, torch.float32, 2),
    (5, 1, 160, True, True, torch.bfloat16, 5),
    (32, 200, 1152, True, False, torch.bfloat16, 1),
    (33, 264, 512, False, False, torch.float32, None),
    (64, 64, 2080, True, True, torch.float32, 10),
    (65, 1024, 1024, True, False, torch.bfloat16, 13),
    (130, 328, 1024, True, False, torch.float32, 64),
    (256, 256, 512, False, False, None, None),
    (300, 520, 640, True, False, torch.float32, 7),
    (515, 776, 1280, True, True, torch.bfloat16, 200),
    (1030, 512, 512, False, False, torch.float32, None),
    (700, 300, 736, True, False, torch.float32, 350),
    (1, 256, 384, True, False, None, None),
    (40, 1032, 896, True, False, torch.bfloat16, 3),
    # a last panel of 32, 64 and 96 elements
    (300, 264, 672, True, False, torch.float32, None),
    (70, 776, 832, False, True, torch.bfloat16, 64),
    (4100, 4104, 736, True, False, torch.float32, 4000),
    # more tiles than workgroups: a workgroup goes from one tile to the next
    (4100, 4360, 512, True, False, torch.float32, 1500),
    (4200, 4104, 640, False, False, torch.bfloat16, 3),
    (4353, 4360, 768, True, False, None, None),
]


@pytest.mark.parametrize("mode, waves, kernel", [k for k in KERNELS if k[1] == 4])
@pytest.mark.parametrize("case", RESIDUAL_CASES, ids=lambda c: "x".join(map(str, c[:3])))
def test_gemm_residual_matches_float64(case, mode, waves, kernel):
    with w4a4_waves(waves), block_kernel(kernel):
        check_residual(case, mode)


def check_residual(case, mode):
    m, n, k, has_bias, gelu, gate_type, rpg = case
    say("residual", case, mode, mxq.block_kernel_name(mode, m, n, k))
    g = gen(m * 31 + n)
    a, w, A, W = quantized(mode, g, m, n, k)
    residual = bf16(randn(g, m, n, scale=2.0))
    bias = bf16(randn(g, n, scale=0.5)) if has_bias else None
    groups = 1 if rpg is None else -(-m // rpg)
    gate = None if gate_type is None else randn(g, groups, n, scale=0.6).to(gate_type)
    to = lambda t: None if t is None else t.to(DEV)
    epi = mxq.EPI_GELU_TANH if gelu else mxq.EPI_NONE
    res_dev = residual.to(DEV)
    y = mxq.gemm_residual(mode, *a, *w, res_dev, bias=to(bias), gate=to(gate), rows_per_group=rpg, epilogue=epi)
    v, err = product(A, W)
    if has_bias:
        v = v + bias.double()
        err = err + 2 * U * v.abs()
    if gelu:
        v, err = gelu64(v), 1.2 * err + 2.0 ** -15 * v.abs()
    f = torch.ones(m, n, dtype=torch.float64) if gate is None else rows_of(gate, m, rpg or m)
    want = residual.double() + f * v
    err = f.abs() * err
    within(y, want, err + BF * (want.abs() + err) + 2 * U * (residual.double().abs() + (f * v).abs()), "y")
    # in place, on the operands' own values
    again = mxq.gemm_residual(mode, *a, *w, res_dev, bias=to(bias), gate=to(gate), rows_per_group=rpg, epilogue=epi, y=res_dev)
    assert again.data_ptr() == res_dev.data_ptr() and torch.equal(again, y)


GATED_CASES = [
    # m, h, k, bias gate, bias up, act
    (1, 32, 32, False, False, mxq.GATED_SILU),
    (1, 1376, 640, True, True, mxq.GATED_GELU_TANH),
    (7, 96, 160, True, False, mxq.GATED_SILU),
    (32, 160, 1152, False, True, mxq.GATED_GELU_TANH),
    (33, 256, 512, False, False, mxq.GATED_SILU),
    (64, 416, 96, True, True, mxq.GATED_SILU),
    (100, 128, 1024, True, True, mxq.GATED_SILU),
    (256, 128, 512, False, False, mxq.GATED_GELU_TANH),
    (300, 384, 640, True, True, mxq.GATED_SILU),
    (515, 416, 1280, True, False, mxq.GATED_GELU_TANH),
    (1030, 640, 512, False, True, mxq.GATED_SILU),
    (350, 160, 736, True, True, mxq.GATED_SILU),
    # a last panel of 32, 64 and 96 elements, of K and of the hidden state
    (300, 288, 672, True, False, mxq.GATED_SILU),
    (70, 192, 832, False, True, mxq.GATED_GELU_TANH),
    (259, 352, 736, True, True, mxq.GATED_SILU),
    (4100, 2144, 1120, False, False, mxq.GATED_SILU),
    # more tiles than workgroups: a workgroup goes from one tile to the next
    (4100, 2176, 512, True, True, mxq.GATED_SILU),
    (4200, 2080, 640, False, False, mxq.GATED_GELU_TANH),
]


@pytest.mark.parametrize("mode, waves, kernel", KERNELS)
@pytest.mark.parametrize("case", GATED_CASES, ids=lambda c: "x".join(map(str, c[:3])))
def test_gemm_gated_matches_float64(case, mode, waves, kernel):
    with w4a4_waves(waves), block_kernel(kernel):
        check_gated(case, mode)


def check_gated(case, mode):
    m, h, k, has_bg, has_bu, act = case
    say("gated", case, mode, mxq.block_kernel_name(mode, m, h, k, gated=True))
    g = gen(m * 17 + h)
    a, w, A, (Wg, Wu) = quantized(mode, g, m, h, k, gated=True)
    bg = bf16(randn(g, h, scale=0.5)) if has_bg else None
    bu = bf16(randn(g, h, scale=0.5)) if has_bu else None
    to = lambda t: None if t is None else t.to(DEV)
    y = mxq.gemm_gated(mode, *a, *w, act, bias_gate=to(bg), bias_up=to(bu))
    gv, ge = product(A, Wg)
    uv, ue = product(A, Wu)
    if has_bg:
        gv = gv + bg.double()
    if has_bu:
        uv = uv + bu.double()
    ge, ue = ge + 2 * U * gv.abs(), ue + 2 * U * uv.abs()
    av = act64(gv, act)
    ae = 1.2 * ge + 2.0 ** -15 * av.abs()
    want = av * uv
    err = ae * (uv.abs() + ue) + av.abs() * ue
    within(y, want, err + BF * (want.abs() + err), "hidden")
    if mode == mxq.W4A4:
        codes, scales = mxq.gemm_gated(mode, *a, *w, act, bias_gate=to(bg), bias_up=to(bu), mxfp4_out=True)
        rc, rs = mxq.quantize_act(mode, y)
        assert_codes_equal(host_u8(scales), host_u8(rs), "hidden scales")
        assert_codes_equal(host_u8(codes), host_u8(rc), "hidden codes")


@pytest.mark.parametrize("h, k", [(32, 32), (96, 160), (160, 512), (4096, 384)])
def test_gated_weight_packing_interleaves_the_rows(h, k):
    g = gen(h + k)
    wg, wu = bf16(randn(g, h, k)).to(DEV), bf16(randn(g, h, k)).to(DEV)
    codes, scales = mxq.quantize_weight_gated_mxfp4(wg, wu)
    both = torch.stack((wg.view(-1, 32, k), wu.view(-1, 32, k)), dim=1).reshape(2 * h, k)
    rc, rs = mxq.quantize_weight_mxfp4(both)
    assert_codes_equal(host_u8(codes), host_u8(rc), "codes")
    assert_codes_equal(host_u8(scales), host_u8(rs), "scales")


@pytest.mark.parametrize("mode, waves, kernel", KERNELS)
@pytest.mark.parametrize("m", [1, 40, 270])
def test_products_write_their_rows_only(mode, waves, kernel, m):
    """Rows before and after the output keep their values."""
    with w4a4_waves(waves), block_kernel(kernel):
        check_rows(mode, m)


def check_rows(mode, m):
    n, k = 256, 512
    g = gen(m)
    a, w, _, _ = quantized(mode, g, m, n, k)
    buf = torch.full((m + 16, n), 7.0, dtype=torch.bfloat16, device=DEV)
    res = bf16(randn(g, m, n)).to(DEV)
    want = mxq.gemm_residual(mode, *a, *w, res)
    mxq.gemm_residual(mode, *a, *w, res, y=buf[8:8 + m])
    assert torch.equal(buf[8:8 + m], want) and (buf[:8] == 7).all() and (buf[8 + m:] == 7).all()
    a, w, _, _ = quantized(mode, g, m, n, k, gated=True)
    want = mxq.gemm_gated(mode, *a, *w, mxq.GATED_SILU)
    buf.fill_(7.0)
    mxq.gemm_gated(mode, *a, *w, mxq.GATED_SILU, y=buf[8:8 + m])
    assert torch.equal(buf[8:8 + m], want) and (buf[:8] == 7).all() and (buf[8 + m:] == 7).all()
    if mode == mxq.W4A4:
        cb = torch.full(((m + 16), n // 2), 9, dtype=torch.uint8, device=DEV)
        sb = torch.full((2 * m * 4 + 64,), 9, dtype=torch.uint8, device=DEV)
        sc = sb[32:32 + 2 * m * 4].view(2, m, 4)
        wc, wsc = mxq.gemm_gated(mode, *a, *w, mxq.GATED_SILU, mxfp4_out=True)
        mxq.gemm_gated(mode, *a, *w, mxq.GATED_SILU, y=cb[8:8 + m], y_scales=sc)
        assert torch.equal(cb[8:8 + m], wc) and torch.equal(sc, wsc)
        assert (cb[:8] == 9).all() and (cb[8 + m:] == 9).all() and (sb[:32] == 9).all() and (sb[32 + 8 * m:] == 9).all()


# ----------------------------------------------------------------- together ----

def block_half(s, mode, stream=None):
    """Feed-forward half of a block: norm, gated projections, second projection into the residual stream."""
    codes, scales, h = mxq.norm_quantize(mode, s["x"], branch=s["branch"], gate=s["gate"], weight=s["weight"],
                                         rows_per_group=s["rpg"], stream=stream)
    if mode == mxq.W4A4:
        hid = mxq.gemm_gated(mode, codes, scales, *s["wg"], mxq.GATED_SILU, mxfp4_out=True, stream=stream)
    else:
        hid = mxq.quantize_act(mode, mxq.gemm_gated(mode, codes, scales, *s["wg"], mxq.GATED_SILU, stream=stream),
                               stream=stream)
    return mxq.gemm_residual(mode, *hid, *s["wd"], h, gate=s["gate"], rows_per_group=s["rpg"], stream=stream), h, hid


def block_state(m, k, h, mode, seed):
    g = gen(seed)
    s = {"x": activation(g, m, k), "branch": bf16(randn(g, m, k)), "weight": bf16(randn(g, k, scale=0.1, mean=1.0)),
         "gate": randn(g, -(-m // 3), k, scale=0.3, mean=0.5)}
    s = {n: v.to(DEV) for n, v in s.items()}
    s["rpg"] = 3
    wg, wu, wd = (bf16(randn(g, *shape, scale=0.05)).to(DEV) for shape in ((h, k), (h, k), (k, h)))
    s["wg"], s["wd"] = mxq.quantize_weight_gated_mxfp4(wg, wu), mxq.quantize_weight_mxfp4(wd)
    return s


@pytest.mark.parametrize("mode", [mxq.W4A4, mxq.W4A8])
@pytest.mark.parametrize("m, k, h", [(1, 640, 1152), (37, 512, 1408), (271, 640, 1152)])
def test_block_half_matches_its_steps(m, k, h, mode):
    """The three operators in a row: each step's result is the definition's on what the step before stored."""
    s = block_state(m, k, h, mode, m)
    y, hs, hid = block_half(s, mode)
    n, _, h2 = mxq.norm_quantize(mxq.POLICY_BF16, s["x"], branch=s["branch"], gate=s["gate"], weight=s["weight"],
                                 rows_per_group=3)
    assert torch.equal(h2, hs)
    gate = rows_of(s["gate"].cpu(), m, 3)
    want_h = s["x"].cpu().double() + gate * s["branch"].cpu().double()
    within(hs, want_h, BF * want_h.abs() + 8 * U * (s["x"].cpu().double().abs() + (gate * s["branch"].cpu().double()).abs()), "h")
    A = decode_act(mode, *hid, m, h)
    v, err = product(A, decode_mxfp4(*s["wd"], k, h))
    want = hs.cpu().double() + gate * v
    err = gate.abs() * err
    within(y, want, err + BF * (want.abs() + err) + 2 * U * (hs.cpu().double().abs() + (gate * v).abs()), "y")
    N = decode_act(mode, *mxq.quantize_act(mode, n), m, k)
    W = decode_mxfp4(*s["wg"], 2 * h, k).view(h // 32, 2, 32, k)
    gv, uv = N @ W[:, 0].reshape(h, k).T, N @ W[:, 1].reshape(h, k).T
    hidden = act64(gv, mxq.GATED_SILU) * uv
    # the quantized hidden state: E2M1 within a quarter of its block's largest value, E4M3 within 2^-4 of the
    # value or half of its smallest step, 2^-10 scales of 1 / 448 of the row's largest
    top = hidden.abs().view(m, -1, 32).amax(2).repeat_interleave(32, 1) if mode == mxq.W4A4 else hidden.abs().amax(1, keepdim=True)
    tol = 0.26 * top if mode == mxq.W4A4 else 0.07 * hidden.abs() + top * 2.0 ** -17 + 0.01 * top
    within(A, hidden, tol + 0.01 * hidden.abs(), "quantized hidden state")


@pytest.mark.parametrize("mode", [mxq.W4A4, mxq.W4A8])
@pytest.mark.parametrize("m", [1, 271])
def test_block_half_captured_replays_like_the_eager_run(m, mode):
    k, h = 640, 1152
    s, other = block_state(m, k, h, mode, 5), block_state(m, k, h, mode, 6)
    want, want_other = block_half(s, mode), block_half(other, mode)
    torch.cuda.synchronize()
    static = {n: v.clone() if isinstance(v, torch.Tensor) else tuple(t.clone() for t in v) if isinstance(v, tuple) else v
              for n, v in s.items()}
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block_half(static, mode)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y, hs, _ = block_half(static, mode)
    for i in range(4):
        src, ref = ((s, want), (other, want_other))[i % 2]
        for name in ("x", "branch", "gate", "weight"):
            static[name].copy_(src[name])
        for name in ("wg", "wd"):
            for to, frm in zip(static[name], src[name]):
                to.copy_(frm)
        graph.replay()
        eager = block_half(src, mode)  # the program's own work between replays
        torch.cuda.synchronize()
        assert torch.equal(y, ref[0]) and torch.equal(hs, ref[1]), f"replay {i}"
        assert torch.equal(eager[0], ref[0])


@pytest.mark.parametrize("mode", [mxq.W4A4, mxq.W4A8])
def test_two_streams_at_once(mode):
    """Calls on two streams at the same time give what each gives alone (no shared scratch)."""
    states = [block_state(m, 640, 1152, mode, m) for m in (9, 300)]
    want = [block_half(s, mode)[0] for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        got.append([block_half(s, mode, stream=st)[0] for s, st in zip(states, streams)])
    torch.cuda.synchronize()
    for pair in got:
        for y, ref in zip(pair, want):
            assert torch.equal(y, ref)


def test_results_do_not_depend_on_the_run():
    s = block_state(45, 640, 1152, mxq.W4A4, 3)
    first = block_half(s, mxq.W4A4)
    for _ in range(3):
        again = block_half(s, mxq.W4A4)
        assert all(torch.equal(a, b) for a, b in zip(first[:2], again[:2]))


def test_empty_problems_write_nothing():
    w = mxq.quantize_weight_mxfp4(torch.zeros(64, 64, dtype=torch.bfloat16, device=DEV))
    wg = mxq.quantize_weight_gated_mxfp4(*(torch.zeros(64, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    for mode in (mxq.W4A4, mxq.W4A8):
        codes, scales, h = mxq.norm_quantize(mode, x, branch=x)
        assert codes.shape[0] == 0 and h.shape == (0, 64)
        y = mxq.gemm_residual(mode, codes, scales, *w, torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
        assert y.shape == (0, 64)
        assert mxq.gemm_gated(mode, codes, scales, *wg, mxq.GATED_SILU).shape == (0, 64)
    torch.cuda.synchronize()


@pytest.mark.parametrize("mode", [mxq.W4A4, mxq.W4A8])
def test_outputs_past_2_gib(mode):
    """The last rows of outputs larger than 2^31 bytes equal the same rows computed alone by the same kernel."""
    m, n, k, last = 140000, 8192, 512, 300
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
    w = mxq.quantize_weight_mxfp4((0.05 * torch.randn(n, k, generator=g, device=DEV)).to(torch.bfloat16))
    wg = mxq.quantize_weight_gated_mxfp4(*((0.05 * torch.randn(n, k, generator=g, device=DEV)).to(torch.bfloat16) for _ in range(2)))
    a, a_last = mxq.quantize_act(mode, x), mxq.quantize_act(mode, x[-last:].contiguous())
    gate = torch.randn(2, n, generator=g, device=DEV)
    residual = torch.randn(m, n, generator=g, device=DEV, dtype=torch.bfloat16)
    assert 2 * m * n > 2 ** 31
    for kernel in ("pipe", "tokens"):
        with block_kernel(kernel):
            say("past 2 GiB", mode, kernel)
            y = mxq.gemm_residual(mode, *a, *w, residual, gate=gate, rows_per_group=m - last)
            part = mxq.gemm_residual(mode, *a_last, *w, residual[-last:], gate=gate[1:])
            assert torch.equal(y[-last:], part)
            del y
            hid = mxq.gemm_gated(mode, *a, *wg, mxq.GATED_SILU)
            assert torch.equal(hid[-last:], mxq.gemm_gated(mode, *a_last, *wg, mxq.GATED_SILU))
            del hid
    h = mxq.norm_quantize(mxq.POLICY_BF16, residual, branch=residual, norm=mxq.NORM_LAYER, h=residual)[0]
    tail = residual[-last:].clone()  # h, in place: twice the residual
    assert torch.equal(h[-last:], mxq.norm_quantize(mxq.POLICY_BF16, tail, norm=mxq.NORM_LAYER)[0])


def test_check_finite_refuses_and_reports(monkeypatch):
    monkeypatch.setenv("MXQ_CHECK_FINITE", "1")
    k = 512
    w = mxq.quantize_weight_mxfp4(bf16(randn(gen(1), 256, k)).to(DEV))
    x = bf16(randn(gen(2), 5, k)).to(DEV)
    bad = x.clone()
    bad[3, 7] = float("inf")
    out = torch.full((5, k), 7.0, dtype=torch.bfloat16, device=DEV)
    for kw in ({"x": bad}, {"x": x, "branch": bad}):
        with pytest.raises(mxq.MxqError) as e:
            mxq.norm_quantize(mxq.POLICY_BF16, out=out, **kw)
        assert e.value.status == mxq.ERR_NONFINITE and (out == 7).all()
    a = mxq.quantize_act(mxq.W4A4, x)
    res = torch.zeros(5, 256, dtype=torch.bfloat16, device=DEV)
    assert torch.isfinite(mxq.gemm_residual(mxq.W4A4, *a, *w, res)).all()
    res[4, 255] = float("nan")
    y = torch.full_like(res, 7.0)
    with pytest.raises(mxq.MxqError) as e:
        mxq.gemm_residual(mxq.W4A4, *a, *w, res, y=y)
    assert e.value.status == mxq.ERR_NONFINITE and (y == 7).all()
    with pytest.raises(mxq.MxqError):
        mxq.quantize_weight_gated_mxfp4(bad.new_full((32, k), float("inf")), bad.new_zeros((32, k)))
