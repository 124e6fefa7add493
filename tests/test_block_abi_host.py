"""The block operators' C ABI and binding on the host: include/mxq_block.h and the library agree, and bad calls are
refused before any HIP call (no GPU needed)."""

import ctypes
import os
import re

import pytest
import torch

import mx_bit_quantized_amd as mxq
from conftest import ROOT
from mx_bit_quantized_amd import block

HEADER = os.path.join(ROOT, "include", "mxq_block.h")
P = 0x10000          # 16-byte aligned, never dereferenced
ODD = 0x10008        # 8-byte aligned only
INF, NAN = float("inf"), float("nan")


def text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_library_exports_every_declared_symbol():
    names = set(re.findall(r"\b(mxq_[a-z0-9_]+)\s*\(", text()))
    assert names == set(block._SIGS)
    for name in names:
        assert hasattr(mxq.lib(), name), name


def test_struct_and_constants_match_the_header():
    body = re.search(r"typedef struct mxq_norm_args \{(.*?)\}", text(), flags=re.S).group(1)
    declared = []
    for stmt in body.split(";"):
        stmt = re.sub(r"\b(const|void|float|int64_t|int32_t)\b|\*", " ", stmt)
        declared += [n.strip() for n in stmt.split(",") if n.strip()]
    assert declared == [n for n, _ in block.NormArgs._fields_]
    assert ctypes.sizeof(block.NormArgs) == 13 * 8 + 7 * 8 + 5 * 4 + 4
    for c, v in (("NORM_NONE", 0), ("NORM_RMS", 1), ("NORM_LAYER", 2), ("GATED_SILU", 0), ("GATED_GELU_TANH", 1)):
        assert re.search(rf"\bMXQ_{c} = {v}\b", text()) and getattr(mxq, c) == v
    assert re.search(rf"define MXQ_NORM_MAX_K {mxq.NORM_MAX_K}\b", text())


def norm(mode=mxq.W4A4, **change):
    a = block.NormArgs()
    base = dict(x=P, branch=P, gate=P, weight=P, scale=P, shift=P, h=P, out=P, out_scales=P, M=4, K=64, ldx=64, ldb=64, ldh=64,
                ld_mod=64, rows_per_group=2, norm=mxq.NORM_RMS, eps=1e-6, branch_scale=1.0)
    base.update(change)
    for n, v in base.items():
        setattr(a, n, v)
    return block._lib().mxq_norm_quantize(mode, ctypes.byref(a), None)


@pytest.mark.parametrize("want, mode, change", [
    (mxq.ERR_MODE, -1, {}), (mxq.ERR_MODE, 4, {}),
    (mxq.ERR_MODE, mxq.W4A4, {"norm": 0}), (mxq.ERR_MODE, mxq.W4A4, {"norm": 3}), (mxq.ERR_MODE, mxq.W4A4, {"post_norm": 3}),
    (mxq.ERR_MODE, mxq.W4A4, {"eps": 0.0}), (mxq.ERR_MODE, mxq.W4A4, {"eps": -1e-6}), (mxq.ERR_MODE, mxq.W4A4, {"eps": INF}),
    (mxq.ERR_MODE, mxq.W4A4, {"eps": NAN}), (mxq.ERR_MODE, mxq.W4A4, {"branch_scale": NAN}),
    (mxq.ERR_MODE, mxq.W4A4, {"mod_type": 2}), (mxq.ERR_MODE, mxq.W4A4, {"post_weight": P}),
    (mxq.ERR_MODE, mxq.W4A4, {"post_bias": P}),
    (mxq.ERR_SHAPE, mxq.W4A4, {"K": 48, "ldx": 64}), (mxq.ERR_SHAPE, mxq.W4A4, {"K": 0}), (mxq.ERR_SHAPE, mxq.W4A4, {"M": -1}),
    (mxq.ERR_SHAPE, mxq.W4A4, {"M": 1 << 31}), (mxq.ERR_SHAPE, mxq.W4A4, {"ldx": 32}), (mxq.ERR_SHAPE, mxq.W4A4, {"ldb": 32}),
    (mxq.ERR_SHAPE, mxq.W4A4, {"ldh": 32}), (mxq.ERR_SHAPE, mxq.W4A4, {"ld_mod": 32}),
    (mxq.ERR_SHAPE, mxq.W4A4, {"rows_per_group": -1}),
    (mxq.ERR_SHAPE, mxq.W4A4, {"K": 32800, "ldx": 32800, "ldb": 32800, "ldh": 32800, "ld_mod": 32800}),
    (mxq.ERR_SHAPE, mxq.POLICY_TRANSFORM_ON, {"act_mult": P}),  # K % 128
    (mxq.ERR_NULL, mxq.POLICY_TRANSFORM_ON, {"K": 128, "ldx": 128, "ldb": 128, "ldh": 128, "ld_mod": 128}),
    (mxq.ERR_NULL, mxq.W4A4, {"x": None}), (mxq.ERR_NULL, mxq.W4A4, {"out": None}), (mxq.ERR_NULL, mxq.W4A4, {"out_scales": None}),
    (mxq.ERR_NULL, mxq.W4A8, {"out_scales": None}),
    (mxq.ERR_NULL, mxq.W4A4, {"branch": None, "h": None}),                      # a gate without a branch
    (mxq.ERR_NULL, mxq.W4A4, {"branch": None, "gate": None}),                   # h without a branch
    (mxq.ERR_NULL, mxq.W4A4, {"branch": None, "gate": None, "h": None, "branch_scale": 0.5}),
    (mxq.ERR_NULL, mxq.W4A4, {"branch": None, "gate": None, "h": None, "post_norm": 1}),
    (mxq.ERR_ALIGN, mxq.W4A4, {"ldx": 68}), (mxq.ERR_ALIGN, mxq.W4A4, {"ldb": 68}), (mxq.ERR_ALIGN, mxq.W4A4, {"ldh": 68}),
    (mxq.ERR_ALIGN, mxq.W4A4, {"ld_mod": 68}),
] + [(mxq.ERR_ALIGN, mxq.W4A4, {n: ODD}) for n in ("x", "branch", "gate", "weight", "bias", "scale", "shift", "h", "out",
                                                   "out_scales", "act_mult")]
    + [(mxq.ERR_ALIGN, mxq.W4A4, {"post_norm": 1, n: ODD}) for n in ("post_weight", "post_bias")])
def test_norm_quantize_refuses(want, mode, change):
    assert norm(mode, **change) == want


def test_norm_quantize_empty_and_null_struct():
    assert norm(M=0, x=None, out=None, out_scales=None) == mxq.OK
    assert block._lib().mxq_norm_quantize(mxq.W4A4, None, None) == mxq.ERR_NULL


def residual(**change):
    a = dict(mode=mxq.W4A4, a=P, asc=P, w=P, wsc=P, bias=P, epi=0, residual=P, gate=P, mod_type=0, ld_mod=64, rpg=2, y=P, M=4, N=64,
             K=64)
    a.update(change)
    return block._lib().mxq_gemm_residual(*a.values(), None)


@pytest.mark.parametrize("want, change", [
    (mxq.ERR_MODE, {"mode": mxq.POLICY_BF16}), (mxq.ERR_MODE, {"mode": mxq.POLICY_TRANSFORM_ON}), (mxq.ERR_MODE, {"epi": 2}),
    (mxq.ERR_MODE, {"mod_type": 2}), (mxq.ERR_SHAPE, {"K": 48}), (mxq.ERR_SHAPE, {"M": -1}), (mxq.ERR_SHAPE, {"N": -1}),
    (mxq.ERR_SHAPE, {"N": 1 << 31}), (mxq.ERR_SHAPE, {"ld_mod": 63}), (mxq.ERR_SHAPE, {"rpg": -1}),
] + [(mxq.ERR_NULL, {n: None}) for n in ("a", "asc", "w", "wsc", "residual", "y")]
    + [(mxq.ERR_ALIGN, {n: ODD}) for n in ("a", "asc", "w", "wsc", "bias", "residual", "gate", "y")])
def test_gemm_residual_refuses(want, change):
    assert residual(**change) == want


def test_gemm_residual_empty():
    none = dict(a=None, asc=None, w=None, wsc=None, residual=None, y=None, bias=None, gate=None)
    assert residual(M=0, **none) == mxq.OK and residual(N=0, **none) == mxq.OK
    # without a gate its type, stride and grouping are not read
    assert residual(M=0, **none, mod_type=9, ld_mod=-1, rpg=-1) == mxq.OK


def gated(**change):
    a = dict(mode=mxq.W4A4, a=P, asc=P, w=P, wsc=P, bg=P, bu=P, act=0, y=P, ysc=P, M=4, H=64, K=64)
    a.update(change)
    return block._lib().mxq_gemm_gated(*a.values(), None)


@pytest.mark.parametrize("want, change", [
    (mxq.ERR_MODE, {"mode": 2}), (mxq.ERR_MODE, {"act": 2}), (mxq.ERR_MODE, {"act": -1}),
    (mxq.ERR_MODE, {"mode": mxq.W4A8}),  # the MXFP4 hidden state belongs to W4A4
    (mxq.ERR_SHAPE, {"K": 16}), (mxq.ERR_SHAPE, {"H": 48}), (mxq.ERR_SHAPE, {"H": -32}), (mxq.ERR_SHAPE, {"H": 1 << 30}),
    (mxq.ERR_SHAPE, {"M": 1 << 31}),
] + [(mxq.ERR_NULL, {n: None}) for n in ("a", "asc", "w", "wsc", "y")]
    + [(mxq.ERR_ALIGN, {n: ODD}) for n in ("a", "asc", "w", "wsc", "bg", "bu", "y", "ysc")])
def test_gemm_gated_refuses(want, change):
    assert gated(**change) == want


def test_gemm_gated_empty():
    none = dict(a=None, asc=None, w=None, wsc=None, bg=None, bu=None, y=None, ysc=None)
    assert gated(M=0, **none) == mxq.OK and gated(H=0, **none) == mxq.OK


@pytest.mark.parametrize("want, args", [
    (mxq.ERR_SHAPE, (P, P, 48, 64, 64, P, P)), (mxq.ERR_SHAPE, (P, P, 64, 48, 64, P, P)), (mxq.ERR_SHAPE, (P, P, 64, 64, 32, P, P)),
    (mxq.ERR_NULL, (None, P, 64, 64, 64, P, P)), (mxq.ERR_NULL, (P, None, 64, 64, 64, P, P)),
    (mxq.ERR_NULL, (P, P, 64, 64, 64, None, P)), (mxq.ERR_NULL, (P, P, 64, 64, 64, P, None)),
    (mxq.ERR_ALIGN, (ODD, P, 64, 64, 64, P, P)), (mxq.ERR_ALIGN, (P, ODD, 64, 64, 64, P, P)),
    (mxq.ERR_ALIGN, (P, P, 64, 64, 68, P, P)), (mxq.OK, (None, None, 0, 64, 64, None, None)),
])
def test_gated_weight_packing_refuses(want, args):
    assert block._lib().mxq_quantize_weight_gated_mxfp4(*args, None) == want


def test_kernel_name_query():
    assert mxq.block_kernel_name(mxq.POLICY_BF16, 1, 64, 64) == "invalid"
    for mode in (mxq.W4A4, mxq.W4A8):
        assert mxq.block_kernel_name(mode, 1, 5120, 13824).startswith("tokens_")
        assert mxq.block_kernel_name(mode, 1, 13824, 5120, gated=True).startswith("tokens_")
        assert mxq.block_kernel_name(mode, 4096, 5120, 160).startswith("tokens_")  # K no multiple of 128


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        mxq.norm_quantize(mxq.W4A4, x)
    with pytest.raises(TypeError):
        mxq.quantize_weight_gated_mxfp4(x, x)
    c = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(TypeError):
        mxq.gemm_gated(mxq.W4A4, c, c, c, c, mxq.GATED_SILU)
    with pytest.raises(TypeError):
        mxq.gemm_residual(mxq.W4A4, c, c, c, c, x)


class FakeCuda(torch.Tensor):
    """A CPU tensor that says it is on a GPU: the binding's checks run, nothing is launched."""
    @staticmethod
    def __new__(cls, t, device="cuda:0"):
        f = torch.Tensor._make_subclass(cls, t)
        f.dev = torch.device(device)
        return f

    is_cuda = property(lambda self: True)
    device = property(lambda self: self.dev)

    def get_device(self):
        return self.dev.index


def fake(*shape, dtype=torch.bfloat16, device="cuda:0"):
    return FakeCuda(torch.zeros(*shape, dtype=dtype), device)


def test_binding_refuses_shapes_devices_and_groups():
    x = fake(6, 64)
    vec = lambda g, n=64, dtype=torch.float32: fake(g, n, dtype=dtype)
    with pytest.raises(ValueError, match="weight is on cuda:1"):
        mxq.norm_quantize(mxq.W4A4, x, weight=fake(64, device="cuda:1"))
    with pytest.raises(ValueError, match="weight must have shape"):
        mxq.norm_quantize(mxq.W4A4, x, weight=fake(32))
    with pytest.raises(TypeError, match="x must have dtype"):
        mxq.norm_quantize(mxq.W4A4, fake(6, 64, dtype=torch.float32))
    with pytest.raises(ValueError, match="do not cover"):
        mxq.norm_quantize(mxq.W4A4, x, scale=vec(2), rows_per_group=2)
    with pytest.raises(ValueError, match="need rows_per_group"):
        mxq.norm_quantize(mxq.W4A4, x, scale=vec(2))
    with pytest.raises(ValueError, match="must share"):
        mxq.norm_quantize(mxq.W4A4, x, scale=vec(2), shift=vec(3), rows_per_group=3)
    with pytest.raises(ValueError, match="must share"):
        mxq.norm_quantize(mxq.W4A4, x, scale=vec(1), shift=vec(1, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="scale must be"):
        mxq.norm_quantize(mxq.W4A4, x, scale=vec(1, 32))
    ac, asc = fake(6, 32, dtype=torch.uint8), fake(1, 6, 4, dtype=torch.uint8)
    wc, wsc = fake(64, 32, dtype=torch.uint8), fake(1, 64, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="residual must have shape"):
        mxq.gemm_residual(mxq.W4A4, ac, asc, wc, wsc, fake(5, 64))
    with pytest.raises(ValueError, match="a_codes must have shape"):
        mxq.gemm_residual(mxq.W4A8, ac, asc, wc, wsc, fake(6, 64))
    with pytest.raises(ValueError, match="bias must have shape"):
        mxq.gemm_residual(mxq.W4A4, ac, asc, wc, wsc, fake(6, 64), bias=fake(63))
    with pytest.raises(ValueError, match="do not cover"):
        mxq.gemm_residual(mxq.W4A4, ac, asc, wc, wsc, fake(6, 64), gate=vec(2), rows_per_group=2)
    with pytest.raises(ValueError, match="bias_up must have shape"):
        mxq.gemm_gated(mxq.W4A4, ac, asc, wc, wsc, mxq.GATED_SILU, bias_up=fake(64))
    with pytest.raises(ValueError, match="w_up must have shape"):
        mxq.quantize_weight_gated_mxfp4(fake(64, 64), fake(32, 64))


def test_binding_refuses_outputs_that_the_call_does_not_write():
    x, h = fake(6, 64), fake(6, 64)
    with pytest.raises(ValueError, match="h is an output"):
        mxq.norm_quantize(mxq.W4A4, x, h=h)
    with pytest.raises(ValueError, match="h is an output"):
        mxq.norm_quantize(mxq.W4A4, x, branch=x, h=h, write_h=False)
    with pytest.raises(ValueError, match="no out_scales"):
        mxq.norm_quantize(mxq.POLICY_BF16, x, out_scales=fake(1, 6, 4, dtype=torch.uint8))


def test_binding_refuses_activations_that_are_no_matrix():
    wc, wsc = fake(64, 32, dtype=torch.uint8), fake(1, 64, 4, dtype=torch.uint8)
    with pytest.raises(TypeError, match="a_codes"):
        mxq.gemm_gated(mxq.W4A4, None, None, wc, wsc, mxq.GATED_SILU)
    with pytest.raises(ValueError, match="a_codes must be 2-D"):
        mxq.gemm_residual(mxq.W4A4, fake(32, dtype=torch.uint8), wsc, wc, wsc, fake(1, 64))
