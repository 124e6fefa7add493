"""Measured cases of the operators around the quantized linears of a transformer block.

Three operators, alone and in the order a block runs them:

* ``norm``      norm_quantize: h = x + gate * branch, its RMS or layer norm, weight and modulation, in bf16 or quantized for
                the next linear;
* ``residual``  gemm_residual: a quantized linear whose epilogue adds bias, GELU, gate and residual;
* ``gated``     gemm_gated: both projections of a gated feed-forward block, the activation and the product;
* ``ffn``       the three of them, with the hidden state and the norm's output quantized in between: the feed-forward half of
                a block, from the attention branch to the block's output.

``own`` chooses between the library's kernels and the plain form, which is elementary torch arithmetic in fp32 on
the same quantized operands. Quantized operands are drawn in bf16 and quantized by the formats' rules: MXFP4 (E2M1 elements,
one power-of-two scale per 32) for weights and W4A4 activations, E4M3 with a scale per token for W4A8 activations.
"""

import math

import torch

own = False  # the library's operators (True) or the plain form (False)

EPS = 1e-6


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one token of a decoder: add the attention branch, norm for the feed-forward block; latency counts
        {"name": "norm token", "op": "norm", "m": 1, "k": 5120, "kind": "rms", "post": False, "gate": "none", "mod": False,
         "groups": 1},
        # a 720p video transformer's self-attention output: gated residual, layer norm, modulated; the largest stream
        {"name": "norm 720p modulated", "op": "norm", "m": 75600, "k": 5120, "kind": "layer", "post": False, "gate": "f32",
         "mod": True, "groups": 1},
        # a batch of prompts with a norm on either side of the block, odd row count and width, bf16 modulation per prompt
        {"name": "norm sandwich batch", "op": "norm", "m": 4099, "k": 4128, "kind": "rms", "post": True, "gate": "bf16",
         "mod": False, "groups": 3},
        # one token through the second projection of a feed-forward block: reads the weights once
        {"name": "residual token w4a4", "op": "residual", "mode": "w4a4", "m": 1, "n": 5120, "k": 13824, "bias": False,
         "gate": "none", "groups": 1, "gelu": False},
        # a few dozen sequences, one token each, through the attention's output projection of a W4A8 block
        {"name": "residual batch w4a8", "op": "residual", "mode": "w4a8", "m": 37, "n": 5120, "k": 5120, "bias": True,
         "gate": "bf16", "groups": 37, "gelu": False},
        # the 480p video transformer's second feed-forward projection into its gated residual stream
        {"name": "residual 480p w4a4", "op": "residual", "mode": "w4a4", "m": 32760, "n": 5120, "k": 13824, "bias": True,
         "gate": "f32", "groups": 1, "gelu": False},
        # one token through both first projections of a gated feed-forward block
        {"name": "gated token w4a4", "op": "gated", "mode": "w4a4", "m": 1, "h": 13824, "k": 5120, "bias": False, "act": "silu"},
        # a text encoder's prompt of 512 tokens, gated GELU, W4A8
        {"name": "gated prompt w4a8", "op": "gated", "mode": "w4a8", "m": 512, "h": 10240, "k": 4096, "bias": False,
         "act": "gelu"},
        # prompts of several sequences together, an odd number of tokens
        {"name": "gated prefill w4a4", "op": "gated", "mode": "w4a4", "m": 8195, "h": 13824, "k": 5120, "bias": True,
         "act": "silu"},
        # a token's way through the whole feed-forward half of a block
        {"name": "ffn token w4a4", "op": "ffn", "mode": "w4a4", "m": 1, "h": 13824, "k": 5120, "act": "silu", "gate": "none"},
        # a small batch of tokens, the same in a W4A8 block
        {"name": "ffn batch w4a8", "op": "ffn", "mode": "w4a8", "m": 16, "h": 10240, "k": 4096, "act": "gelu", "gate": "none"},
        # a prompt's way through it
        {"name": "ffn prompt w4a4", "op": "ffn", "mode": "w4a4", "m": 4095, "h": 13824, "k": 5120, "act": "silu",
         "gate": "f32"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "residual", "gated", "ffn"])
    if op == "norm":
        m = _spread(rng, 1, 40000)
        return {"op": op, "m": m, "k": 32 * _spread(rng, 4, 256), "kind": rng.choice(["rms", "layer"]),
                "post": rng.random() < 0.3, "gate": rng.choice(["none", "f32", "bf16"]), "mod": rng.random() < 0.5,
                "groups": rng.randint(1, min(4, m))}
    mode = rng.choice(["w4a4", "w4a8"])
    m = _spread(rng, 1, 6000)
    k = 32 * _spread(rng, 16, 216)
    if op == "residual":
        return {"op": op, "mode": mode, "m": m, "n": 8 * _spread(rng, 40, 1000) + rng.choice([0, 0, 0, 1, 4]), "k": k,
                "bias": rng.random() < 0.5, "gate": rng.choice(["none", "f32", "bf16"]), "groups": rng.randint(1, min(4, m)),
                "gelu": rng.random() < 0.2}
    h = 32 * _spread(rng, 20, 432)
    if op == "gated":
        return {"op": op, "mode": mode, "m": m, "h": h, "k": k, "bias": rng.random() < 0.5, "act": rng.choice(["silu", "gelu"])}
    return {"op": op, "mode": mode, "m": m, "h": h, "k": k, "act": rng.choice(["silu", "gelu"]),
            "gate": rng.choice(["none", "f32", "bf16"])}


def _mod_bytes(gate):
    return {"none": 0, "bf16": 2, "f32": 4}[gate]


def _act_bytes(mode, m, k):  # codes and scales of a quantized activation
    return m * k * 17 / 32 if mode == "w4a4" else m * (k + 4)


def work(case):
    m, k = case["m"], case["k"]
    if case["op"] == "norm":
        vec = k * (2 + (2 if case["post"] else 0) + case["groups"] * (_mod_bytes(case["gate"]) + (8 if case["mod"] else 0)))
        return {"bytes": 8 * m * k + vec, "flops": (12 + (6 if case["post"] else 0)) * m * k}
    if case["op"] == "residual":
        n = case["n"]
        return {"bytes": _act_bytes(case["mode"], m, k) + n * k * 17 / 32 + 4 * m * n + (2 * n if case["bias"] else 0)
                + case["groups"] * n * _mod_bytes(case["gate"]), "flops": 2 * m * n * k}
    h = case["h"]
    if case["op"] == "gated":
        return {"bytes": _act_bytes(case["mode"], m, k) + 2 * h * k * 17 / 32 + 2 * m * h + (4 * h if case["bias"] else 0),
                "flops": 4 * m * h * k}
    return {"bytes": 8 * m * k + 3 * h * k * 17 / 32 + 2 * k + k * _mod_bytes(case["gate"]), "flops": 6 * m * h * k}


# ----------------------------------------------------------------- inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activation(g, m, k):
    """Normal values with one channel in 200 ten times as large, as transformers' activations have."""
    x = _randn(g, m, k)
    x[:, torch.randperm(k, generator=g, device="cuda")[: max(1, k // 200)]] *= 10.0
    return x.to(torch.bfloat16)


def _vector(g, n, mean, std):
    return (mean + std * _randn(g, n)).to(torch.bfloat16)


def _modulation(g, kind, groups, n, mean, std):
    if kind == "none":
        return None
    return (mean + std * _randn(g, groups, n)).to(torch.float32 if kind == "f32" else torch.bfloat16)


def _inputs(case, seed):
    """The tensors of a case in bf16 (modulation: its own type), before anything is quantized."""
    g, m, k, t = _gen(seed), case["m"], case["k"], {}
    if case["op"] == "norm":
        t["x"], t["branch"] = _activation(g, m, k), _randn(g, m, k).to(torch.bfloat16)
        t["weight"] = _vector(g, k, 1.0, 0.1)
        t["post_weight"] = _vector(g, k, 0.5, 0.1) if case["post"] else None
        t["gate"] = _modulation(g, case["gate"], case["groups"], k, 0.5, 0.3)
        kind = "bf16" if case["gate"] == "bf16" else "f32"  # the modulation vectors of a block share their type
        t["scale"] = _modulation(g, kind, case["groups"], k, 0.0, 0.2) if case["mod"] else None
        t["shift"] = _modulation(g, kind, case["groups"], k, 0.0, 0.2) if case["mod"] else None
    elif case["op"] == "residual":
        n = case["n"]
        t["a"] = _activation(g, m, k)
        t["w"] = (0.02 * _randn(g, n, k)).to(torch.bfloat16)
        t["bias"] = _vector(g, n, 0.0, 0.1) if case["bias"] else None
        t["gate"] = _modulation(g, case["gate"], case["groups"], n, 0.5, 0.3)
        t["residual"] = (2.0 * _randn(g, m, n)).to(torch.bfloat16)
    else:
        h = case["h"]
        if case["op"] == "gated":
            t["a"] = _activation(g, m, k)
            t["bias_gate"] = _vector(g, h, 0.0, 0.1) if case["bias"] else None
            t["bias_up"] = _vector(g, h, 0.0, 0.1) if case["bias"] else None
        else:
            t["x"], t["branch"] = _activation(g, m, k), _randn(g, m, k).to(torch.bfloat16)
            t["weight"] = _vector(g, k, 1.0, 0.1)
            t["gate"] = _modulation(g, case["gate"], 1, k, 0.5, 0.3)
            t["w_down"] = (0.02 * _randn(g, k, h)).to(torch.bfloat16)
        t["w_gate"] = (0.02 * _randn(g, h, k)).to(torch.bfloat16)
        t["w_up"] = (0.02 * _randn(g, h, k)).to(torch.bfloat16)
    return t


def _rows_per_group(case):
    return -(-case["m"] // case.get("groups", 1))


def prepare(case, seed):
    """Inputs, with the weights packed and (where the operator takes them quantized) the activations quantized: a program has
    the former from its start and the latter from the operator before. Each side keeps them in its own layout."""
    t = _inputs(case, seed)
    s = {"case": case, "rpg": _rows_per_group(case)}
    if own:
        import mx_bit_quantized_amd as mxq

        mode = mxq.W4A8 if case.get("mode") == "w4a8" else mxq.W4A4
        s["mode"] = mode
        if "a" in t:
            s["a"] = mxq.quantize_act(mode, t.pop("a"))
        if "w" in t:
            s["w"] = mxq.quantize_weight_mxfp4(t.pop("w"))
        if "w_down" in t:
            s["w_down"] = mxq.quantize_weight_mxfp4(t.pop("w_down"))
        if "w_gate" in t:
            s["w_gated"] = mxq.quantize_weight_gated_mxfp4(t.pop("w_gate"), t.pop("w_up"))
    else:
        if "a" in t:
            s["a"] = _mxfp4(t.pop("a").float()) if case["mode"] == "w4a4" else _e4m3(t.pop("a").float())
        for name in ("w", "w_down", "w_gate", "w_up"):
            if name in t:
                s[name] = _mxfp4(t.pop(name).float())
    s.update(t)
    return s


# ------------------------------------------------------------------- runs ----

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import mx_bit_quantized_amd as mxq

    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        n, _, h = mxq.norm_quantize(mxq.POLICY_BF16, s["x"], branch=s["branch"], gate=s["gate"],
                                    norm=mxq.NORM_RMS if case["kind"] == "rms" else mxq.NORM_LAYER,
                                    post_norm=mxq.NORM_RMS if case["post"] else mxq.NORM_NONE, post_weight=s["post_weight"],
                                    weight=s["weight"], scale=s["scale"], shift=s["shift"], rows_per_group=s["rpg"], eps=EPS)
        return n, h
    if op == "residual":
        return mxq.gemm_residual(s["mode"], *s["a"], *s["w"], s["residual"], bias=s["bias"], gate=s["gate"],
                                 rows_per_group=s["rpg"], epilogue=mxq.EPI_GELU_TANH if case["gelu"] else mxq.EPI_NONE)
    act = mxq.GATED_SILU if case["act"] == "silu" else mxq.GATED_GELU_TANH
    if op == "gated":
        return mxq.gemm_gated(s["mode"], *s["a"], *s["w_gated"], act, bias_gate=s["bias_gate"], bias_up=s["bias_up"])
    codes, scales, h = mxq.norm_quantize(s["mode"], s["x"], branch=s["branch"], weight=s["weight"], eps=EPS)
    if s["mode"] == mxq.W4A4:
        hidden = mxq.gemm_gated(s["mode"], codes, scales, *s["w_gated"], act, mxfp4_out=True)
    else:
        hidden = mxq.quantize_act(s["mode"], mxq.gemm_gated(s["mode"], codes, scales, *s["w_gated"], act))
    return mxq.gemm_residual(s["mode"], *hidden, *s["w_down"], h, gate=s["gate"]), h


# ------------------------------------------------------------- plain form ----

def _mxfp4(v):
    """fp32 [rows, K] -> (codes [rows, K] uint8: sign * 8 + magnitude index, block exponents [rows, K / 32])."""
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(dim=2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32)).clamp(-127, 127)
    r = torch.ldexp(b.abs(), -e[..., None])  # in units of the block's scale, below 8
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
    q = (torch.round(r / step) * step).clamp_(max=6.0)
    index = torch.where(q < 2, 2 * q, torch.where(q < 4, q + 2, q / 2 + 4))
    return (index + 8 * torch.signbit(b)).to(torch.uint8).view(v.shape), e


def _of_mxfp4(codes, e):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = table[codes.int()].view(codes.shape[0], -1, 32)
    return torch.ldexp(v, e[..., None]).view(codes.shape)


def _e4m3(v):
    amax = v.abs().amax(dim=1, keepdim=True)
    s = amax / torch.full_like(amax, 448.0)  # (a Python number would be multiplied by its rounded reciprocal)
    q = torch.where(s > 0, v / s, torch.zeros_like(v)).clamp(-448.0, 448.0)
    return q.to(torch.float8_e4m3fn), s


def _operand(case, pair):
    return _of_mxfp4(*pair) if pair[0].dtype == torch.uint8 else pair[0].float() * pair[1]


def _bf16(v):
    return v.to(torch.bfloat16).float()


def _rows(v, m, rpg):
    """A modulation vector's row for each of m rows."""
    return None if v is None else v.float()[torch.arange(m, device=v.device) // rpg]


def _normed(v, kind):
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    return v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)


def _activated(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _run_plain(s):
    case, op, m = s["case"], s["case"]["op"], s["case"]["m"]
    if op == "norm":
        b = s["branch"].float()
        if case["post"]:
            b = _normed(b, "rms") * s["post_weight"].float()
        if s["gate"] is not None:
            b = b * _rows(s["gate"], m, s["rpg"])
        h = (s["x"].float() + b).to(torch.bfloat16)
        n = _normed(h.float(), case["kind"]) * s["weight"].float()
        if case["mod"]:
            n = n * (1 + _rows(s["scale"], m, s["rpg"])) + _rows(s["shift"], m, s["rpg"])
        return n.to(torch.bfloat16), h
    if op == "residual":
        y = _operand(case, s["a"]) @ _of_mxfp4(*s["w"]).t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        if case["gelu"]:
            y = _activated(y, "gelu")
        if s["gate"] is not None:
            y = y * _rows(s["gate"], m, s["rpg"])
        return (y + s["residual"].float()).to(torch.bfloat16)
    if op == "gated":
        a = _operand(case, s["a"])
        g, u = a @ _of_mxfp4(*s["w_gate"]).t(), a @ _of_mxfp4(*s["w_up"]).t()
        if s["bias_gate"] is not None:
            g, u = g + s["bias_gate"].float(), u + s["bias_up"].float()
        return (_activated(g, case["act"]) * u).to(torch.bfloat16)
    quant = _mxfp4 if case["mode"] == "w4a4" else _e4m3
    h = (s["x"].float() + s["branch"].float()).to(torch.bfloat16)
    a = _operand(case, quant(_bf16(_normed(h.float(), "rms") * s["weight"].float())))
    hid = _activated(a @ _of_mxfp4(*s["w_gate"]).t(), case["act"]) * (a @ _of_mxfp4(*s["w_up"]).t())
    y = _operand(case, quant(_bf16(hid))) @ _of_mxfp4(*s["w_down"]).t()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    return (y + h.float()).to(torch.bfloat16), h


# ---------------------------------------------------- definition in 64 bits ----

# E2M1's values and the borders between them; a value on a border goes to the neighbour of even code
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


def _exact_mxfp4(v):
    """The values that MXFP4 gives to float64 [rows, K] holding bf16 values."""
    out = torch.empty_like(v)
    for r0 in range(0, v.shape[0], 4096):  # a few thousand rows at a time: the comparisons are eight times the input's size
        b = v[r0:r0 + 4096].reshape(-1, 32)
        top = b.abs().amax(dim=1, keepdim=True)
        scale = torch.exp2(torch.floor(torch.log2(top)).clamp(-125, 129) - 2)
        r = b.abs() / scale
        code = torch.zeros_like(b, dtype=torch.int64)
        for i, border in enumerate(_BORDERS):
            code += (r > border) | ((r == border) & (i % 2 == 1))
        out[r0:r0 + 4096] = (torch.tensor(_E2M1, device=v.device, dtype=torch.float64)[code] * scale * torch.sign(b)) \
            .view(-1, v.shape[1])
    return out


def _exact_e4m3(v):
    """The values that E4M3 with a scale per row gives: the quotient is an fp32 one by the format's rule."""
    s = (v.abs().amax(dim=1, keepdim=True).float() / torch.tensor(448.0, device=v.device)).double()
    r = (v.float() / torch.where(s > 0, s, torch.ones_like(s)).float()).double()
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.clamp(torch.round(r / step) * step, -448.0, 448.0) * s


def _exact_operand(case, v):
    return _exact_mxfp4(v) if case["mode"] == "w4a4" else _exact_e4m3(v)


def _exact_act(v, act):
    if act == "silu":
        return v * torch.special.expit(v)
    return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))


def _exact_norm(v, kind):
    if kind == "layer":
        return (v - v.mean(1, keepdim=True)) / torch.sqrt(v.var(1, unbiased=False, keepdim=True) + EPS)
    return v / torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + EPS)


def _exact_spread(v, case):
    rpg = _rows_per_group(case)
    return v.double().repeat_interleave(rpg, dim=0)[: case["m"]]


def exact(case, seed):
    t = {k: v if v is None or k in ("gate", "scale", "shift") else v.double() for k, v in _inputs(case, seed).items()}
    op = case["op"]
    if op == "norm":
        b = t["branch"]
        if case["post"]:
            b = _exact_norm(b, "rms") * t["post_weight"]
        h = t["x"] + (b if t["gate"] is None else b * _exact_spread(t["gate"], case))
        n = _exact_norm(h.to(torch.bfloat16).double(), case["kind"]) * t["weight"]  # the norm is taken of the stored h
        if case["mod"]:
            n = n * (1 + _exact_spread(t["scale"], case)) + _exact_spread(t["shift"], case)
        return n, h
    if op == "residual":
        y = torch.matmul(_exact_operand(case, t["a"]), _exact_mxfp4(t["w"]).t().contiguous())
        if t["bias"] is not None:
            y += t["bias"]
        if case["gelu"]:
            y = _exact_act(y, "gelu")
        return t["residual"] + (y if t["gate"] is None else y * _exact_spread(t["gate"], case))
    w_gate, w_up = (_exact_mxfp4(t.pop(k)).t().contiguous() for k in ("w_gate", "w_up"))
    if op == "gated":
        a = _exact_operand(case, t["a"])
        g, u = torch.matmul(a, w_gate), torch.matmul(a, w_up)
        if t["bias_gate"] is not None:
            g, u = g + t["bias_gate"], u + t["bias_up"]
        return _exact_act(g, case["act"]) * u
    h = t["x"] + t["branch"]
    a = _exact_operand(case, (_exact_norm(h.to(torch.bfloat16).double(), "rms") * t["weight"]).to(torch.bfloat16).double())
    hid = _exact_act(torch.matmul(a, w_gate), case["act"]) * torch.matmul(a, w_up)
    y = torch.matmul(_exact_operand(case, hid.to(torch.bfloat16).double()), _exact_mxfp4(t["w_down"]).t().contiguous())
    if t["gate"] is not None:
        y = y * _exact_spread(t["gate"], dict(case, groups=1))
    return y + h.to(torch.bfloat16).double(), h
