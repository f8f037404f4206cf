"""The feed-forward operators of language models on their real range of sizes:
the gated product (both projections, the activation and the product), its
gradients, microscaled 4-bit quantisation, and products of microscaled operands.

``run`` computes them in plain torch operations in 32 bits, or, where ``own``
is true, through the library's entry points. ``exact`` is their definition in
64 bits.
"""
import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    ffn = {"op": "ffn", "act": "silu", "linear": True, "keep": False, "pad": 0}
    grad = {"op": "ffn_grad", "act": "silu", "linear": True, "recompute": False, "pad": 0}
    quant = {"op": "quantize", "pad": 0}
    gemm = {"op": "mx_gemm", "act": "none", "alpha": 1.0, "pad": 0}
    return [
        # One token of one request: the weights are read once, latency and bandwidth count.
        {"name": "ffn token 1x4096x16384", **ffn, "rows": 1, "width": 4096, "hidden": 16384, "type": "bf16"},
        # A decoding batch, weights stored input by output.
        {"name": "ffn batch 48x2048x8192", **ffn, "rows": 48, "width": 2048, "hidden": 8192, "type": "fp16",
         "act": "gelu_tanh", "linear": False},
        # A long prompt or the forward pass of evaluation.
        {"name": "ffn prompt 8192x4096x16384", **ffn, "rows": 8192, "width": 4096, "hidden": 16384, "type": "bf16"},
        # A training step's forward pass with odd sizes and padded strides, pre-activations kept.
        {"name": "ffn train 2047x1000x2501", **ffn, "rows": 2047, "width": 1000, "hidden": 2501, "type": "fp16",
         "act": "gelu", "keep": True, "pad": 3},
        # A training step's gradients from the pre-activations kept.
        {"name": "ffn grad 4096x4096x8192", **grad, "rows": 4096, "width": 4096, "hidden": 8192, "type": "bf16"},
        # The same with the pre-activations computed again instead of kept, weights stored input by output.
        {"name": "ffn regrad 8192x2048x8192", **grad, "rows": 8192, "width": 2048, "hidden": 8192, "type": "bf16",
         "linear": False, "recompute": True},
        # A small micro-batch of odd sizes.
        {"name": "ffn grad 515x1001x2003", **grad, "rows": 515, "width": 1001, "hidden": 2003, "type": "fp16",
         "act": "gelu_tanh"},
        # Weights or a long prompt's activations brought to four bits and back.
        {"name": "quantize 8192x8192", **quant, "rows": 8192, "width": 8192, "type": "bf16"},
        # A decoding batch's activations, an odd width and stride.
        {"name": "quantize 33x5001 fp32", **quant, "rows": 33, "width": 5001, "type": "fp32", "pad": 3},
        # One token through a projection held in four bits: the activations are quantised on the way.
        {"name": "mx token 1x8192x8192", **gemm, "rows": 1, "cols": 8192, "width": 8192, "type": "bf16", "out": "bf16"},
        # A long prompt through a projection.
        {"name": "mx prompt 8192x8192x8192", **gemm, "rows": 8192, "cols": 8192, "width": 8192, "type": "bf16",
         "out": "bf16"},
        # The gated product of a prompt with an odd number of rows, in four bits.
        {"name": "mx gated 2049x4096x8200", **gemm, "rows": 2049, "cols": 8200, "width": 4096, "type": "fp16",
         "out": "fp16", "act": "silu"},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):  # half of them multiples of 64, as models have them
        n = size(lo, hi)
        return n if rng.random() < 0.5 else max(64, n // 64 * 64)

    def capped(n, most):
        return max(1, min(n, most))

    op = rng.choice(["ffn", "ffn_grad", "quantize", "mx_gemm"])
    pad = rng.choice([0, 0, 8, 3])
    half = rng.choice(["bf16", "fp16"])
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    if op == "ffn":
        k, f = width(64, 8192), width(64, 16384)
        return {"op": op, "act": act, "linear": rng.random() < 0.5, "keep": rng.random() < 0.5, "pad": pad,
                "rows": capped(size(1, 8192), 2**38 // (k * f)), "width": k, "hidden": f, "type": half}
    if op == "ffn_grad":
        k, f = width(64, 8192), width(64, 16384)
        return {"op": op, "act": act, "linear": rng.random() < 0.5, "recompute": rng.random() < 0.5, "pad": pad,
                "rows": capped(size(1, 8192), 2**37 // (k * f)), "width": k, "hidden": f, "type": half}
    if op == "quantize":
        k = width(32, 16384)
        return {"op": op, "pad": pad, "rows": capped(size(1, 65536), 2**26 // k), "width": k,
                "type": rng.choice(["bf16", "fp16", "fp32"])}
    k, n = width(64, 16384), width(64, 16384)
    return {"op": op, "act": rng.choice(["none", "none", "silu", "gelu_tanh"]), "alpha": rng.choice([1.0, 0.125]), "pad": pad,
            "rows": capped(size(1, 8192), 2**38 // (k * n)), "cols": n, "width": k, "type": half,
            "out": rng.choice(["bf16", "fp16", "fp32"])}


# ---- inputs -------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"ffn": _prepare_ffn, "ffn_grad": _prepare_grad, "quantize": _prepare_quantize,
            "mx_gemm": _prepare_gemm}[case["op"]](case, g)


def _empty(rows, width, dtype, pad):
    return torch.empty(rows, width + pad, device="cuda", dtype=dtype)[:, :width]


def _randn(g, rows, width, dtype, pad=0, scale=1.0):
    x = _empty(rows, width, dtype, pad)
    x.copy_(torch.randn(rows, width, device="cuda", generator=g).mul_(scale))
    return x


def _prepare_ffn(case, g):
    m, k, f, pad, dtype = case["rows"], case["width"], case["hidden"], case["pad"], _TYPES[case["type"]]
    s = {"case": case, "x": _randn(g, m, k, dtype, pad)}
    s["w"] = _randn(g, 2 * f, k, dtype, pad, k**-0.5) if case["linear"] else _randn(g, k, 2 * f, dtype, pad, k**-0.5)
    s["h"] = _empty(m, f, dtype, pad)
    if case["keep"]:
        s["preact"] = _empty(m, 2 * f, dtype, pad)
    return s


def _prepare_grad(case, g):
    s = _prepare_ffn({**case, "keep": not case["recompute"]}, g)
    m, k, f, pad, dtype = case["rows"], case["width"], case["hidden"], case["pad"], _TYPES[case["type"]]
    s["case"] = case
    del s["h"]
    if "preact" in s:  # what the forward pass kept
        s["preact"].copy_(s["x"] @ (s["w"].t() if case["linear"] else s["w"]))
    s["dh"] = _randn(g, m, f, dtype, pad)
    s["dx"], s["dw"] = _empty(m, k, dtype, pad), _empty(*s["w"].shape, dtype, pad)
    return s


def _activations(g, rows, width, dtype, pad):
    """Normal values with a few large columns, as the inputs of a model's products have them."""
    x = torch.randn(rows, width, device="cuda", generator=g)
    x[:, ::37] *= 8.0
    out = _empty(rows, width, dtype, pad)
    return out.copy_(x)


def _prepare_quantize(case, g):
    rows, width = case["rows"], case["width"]
    s = {"case": case, "x": _activations(g, rows, width, _TYPES[case["type"]], case["pad"])}
    s["values"] = torch.empty(rows, width, device="cuda", dtype=s["x"].dtype)
    s.update(_storage(rows, width, ""))
    return s


def _storage(rows, width, name):
    """Room for a microscaled matrix: two codes a byte, 16 bytes for 32 columns; scales in tiles of 128 rows by 4 blocks."""
    return {name + "codes": torch.zeros(rows, -(-width // 32) * 16, device="cuda", dtype=torch.uint8),
            name + "scales": torch.zeros(-(-rows // 128), -(-width // 128), 32, 4, 4, device="cuda", dtype=torch.uint8)}


def _weights(g, rows, width, name):
    """A weight matrix that was quantised beforehand."""
    s = _storage(rows, width, name)
    w = torch.randn(rows, width, device="cuda", generator=g).mul_(width**-0.5)
    code, e = _quantized(w)
    pair = code.view(rows, -1, 2)
    s[name + "codes"].copy_(pair[:, :, 0] | (pair[:, :, 1] << 4))
    whole = torch.zeros(s[name + "scales"].shape[0] * 128, s[name + "scales"].shape[1] * 4, device="cuda", dtype=torch.uint8)
    whole[:rows, :e.shape[1]] = e
    # Row r = 128 i + 32 j + l, block 4 c + b: tile (i, c), byte 16 l + 4 j + b.
    s[name + "scales"].copy_(whole.view(-1, 4, 32, whole.shape[1] // 4, 4).permute(0, 3, 2, 1, 4))
    return s


def _prepare_gemm(case, g):
    m, n, k = case["rows"], case["cols"], case["width"]
    s = {"case": case, "x": _activations(g, m, k, _TYPES[case["type"]], case["pad"])}
    s.update(_weights(g, n, k, "w_"))
    if case["act"] != "none":
        s.update(_weights(g, n, k, "u_"))
    s.update(_storage(m, k, "x_"))
    s["out"] = _empty(m, n, _TYPES[case["out"]], case["pad"])
    return s


# ---- one pass -------------------------------------------------------------------


def run(state):
    case = state["case"]
    if own:
        return _own(state)
    return {"ffn": _plain_ffn, "ffn_grad": _plain_grad, "quantize": _plain_quantize, "mx_gemm": _plain_gemm}[case["op"]](state)


def _own(s):
    import shape_adaptive_tile_gb300 as sat

    case, stream = s["case"], torch.cuda.current_stream().cuda_stream
    if "call" not in s:  # the argument blocks that a program keeps beside its buffers
        s["call"] = {"ffn": _ffn_call, "ffn_grad": _grad_call, "quantize": _quantize_call, "mx_gemm": _gemm_call}[case["op"]](sat, s)
    if case["op"] == "ffn":
        sat.check(sat.ffn_gated(s["call"], stream))
        return {n: s[n] for n in ("h", "preact") if n in s}
    if case["op"] == "ffn_grad":
        sat.check(sat.ffn_gated_backward(*s["call"], stream))
        return {"dx": s["dx"], "dw": s["dw"]}
    if case["op"] == "quantize":
        sat.check(sat.mxfp4_quantize(s["call"][0], stream))
        sat.check(sat.mxfp4_dequantize(s["call"][1], stream))
        return {"values": s["values"]}
    sat.check(sat.mxfp4_quantize(s["call"][0], stream))
    sat.check(sat.mxfp4_gemm(s["call"][1], stream))
    return {"out": s["out"]}


def _ffn_args(sat, s):
    case = s["case"]
    return sat.FfnArgs(
        rows=case["rows"], width=case["width"], hidden=case["hidden"], type=case["type"], activation=case["act"],
        w_by_output=int(case["linear"]), x=s["x"], ldx=s["x"].stride(0), w=s["w"], ldw=s["w"].stride(0), h=s.get("h"),
        ldh=s["h"].stride(0) if "h" in s else 0, preact=s.get("preact"),
        ldp=s["preact"].stride(0) if "preact" in s else 0)


def _ffn_call(sat, s):
    args = _ffn_args(sat, s)
    size = sat.ffn_gated_workspace(args)
    if size:
        args.workspace, args.workspace_bytes = torch.empty(size, device="cuda", dtype=torch.uint8), size
    return args


def _grad_call(sat, s):
    args = _ffn_args(sat, s)
    grads = sat.FfnGrads(dh=s["dh"], lddh=s["dh"].stride(0), dx=s["dx"], lddx=s["dx"].stride(0), dw=s["dw"],
                         lddw=s["dw"].stride(0), dw_type=s["case"]["type"])
    size = sat.ffn_gated_backward_workspace(args, grads)
    grads.workspace, grads.workspace_bytes = torch.empty(size, device="cuda", dtype=torch.uint8), size
    return args, grads


def _quantized_args(sat, s, name, rows, width, kind, values):
    return sat.Mxfp4Args(rows=rows, width=width, type=kind, values=values, ldv=values.stride(0), codes=s[name + "codes"],
                         ldc=s[name + "codes"].stride(0), scales=s[name + "scales"])


def _quantize_call(sat, s):
    case = s["case"]
    return tuple(_quantized_args(sat, s, "", case["rows"], case["width"], case["type"], s[v]) for v in ("x", "values"))


def _gemm_call(sat, s):
    case = s["case"]
    x = _quantized_args(sat, s, "x_", case["rows"], case["width"], case["type"], s["x"])
    up = {} if case["act"] == "none" else {"up_codes": s["u_codes"], "ldu": s["u_codes"].stride(0), "up_scales": s["u_scales"]}
    return x, sat.Mxfp4GemmArgs(
        rows=case["rows"], cols=case["cols"], width=case["width"], out_type=case["out"], activation=case["act"],
        alpha=case["alpha"], a_codes=s["x_codes"], lda=s["x_codes"].stride(0), a_scales=s["x_scales"], b_codes=s["w_codes"],
        ldb=s["w_codes"].stride(0), b_scales=s["w_scales"], out=s["out"], ldo=s["out"].stride(0), **up)


_ROOT_2_OVER_PI = math.sqrt(2.0 / math.pi)


def _act(g, kind):
    """(activation, its derivative) of g."""
    if kind == "none":
        return g, torch.ones_like(g)
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = torch.tanh(_ROOT_2_OVER_PI * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _ROOT_2_OVER_PI * (1.0 + 0.134145 * g * g)
    return torch.where(g > 0, g, 0.0), torch.where(g > 0, 1.0, 0.0)


def _plain_ffn(s):
    case = s["case"]
    w = s["w"].float()
    z = s["x"].float() @ (w.t() if case["linear"] else w)
    g, u = z[:, :case["hidden"]], z[:, case["hidden"]:]
    s["h"].copy_(_act(g, case["act"])[0] * u)
    if not case["keep"]:
        return {"h": s["h"]}
    s["preact"].copy_(z)
    return {"h": s["h"], "preact": s["preact"]}


def _plain_grad(s):
    case, f = s["case"], s["case"]["hidden"]
    x, w, dh = s["x"].float(), s["w"].float(), s["dh"].float()
    z = x @ (w.t() if case["linear"] else w) if case["recompute"] else s["preact"].float()
    g, u = z[:, :f], z[:, f:]
    a, da = _act(g, case["act"])
    dz = torch.cat([dh * u * da, dh * a], 1)
    if case["linear"]:
        s["dx"].copy_(dz @ w)
        s["dw"].copy_(dz.t() @ x)
    else:
        s["dx"].copy_(dz @ w.t())
        s["dw"].copy_(x.t() @ dz)
    return {"dx": s["dx"], "dw": s["dw"]}


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantized(x):
    """(codes, biased scale exponents) of the rows of x, 32 columns to a block, the last block filled up with zeros."""
    rows, width = x.shape
    blocks = -(-width // 32)
    v = torch.zeros(rows, blocks * 32, device="cuda")
    v[:, :width] = x.float()
    v = v.view(rows, blocks, 32)
    top = v.abs().amax(-1)
    # frexp: top = m 2^e with m in [0.5, 1), so floor(log2 top) is e - 1; the largest power of e2m1 is 2^2.
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
    v = _times_power(v, -e)
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code | ((v < 0).to(torch.uint8) << 3)).view(rows, blocks * 32), (e + 127).to(torch.uint8)


def _times_power(v, e):
    """v 2^e for each block, exactly: the powers from their bits, in two steps, as 2^-127 is not a normal 32-bit float."""
    for n in (e // 2, e - e // 2):
        v = v * ((n.int() + 127) << 23).view(torch.float32)[:, :, None]
    return v


def _valued(code, e):
    """The values in 32 bits of codes and biased exponents."""
    v = torch.tensor(_E2M1, device="cuda")[(code & 7).long()]
    v = torch.where(code > 7, -v, v).view(*e.shape, 32)
    return _times_power(v, e.int() - 127).flatten(1)


def _plain_quantize(s):
    s["values"].copy_(_valued(*_quantized(s["x"]))[:, :s["case"]["width"]])
    return {"values": s["values"]}


def _stored(s, name, rows):
    """The values in 32 bits of a stored matrix."""
    codes, scales = s[name + "codes"], s[name + "scales"]
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(1)
    e = scales.permute(0, 3, 2, 1, 4).reshape(scales.shape[0] * 128, -1)
    return _valued(code, e[:rows, :codes.shape[1] // 16])


def _plain_gemm(s):
    case = s["case"]
    x = _valued(*_quantized(s["x"]))
    z = case["alpha"] * (x @ _stored(s, "w_", case["cols"]).t())
    if case["act"] != "none":
        z = _act(z, case["act"])[0] * (case["alpha"] * (x @ _stored(s, "u_", case["cols"]).t()))
    s["out"].copy_(z)
    return {"out": s["out"]}


# ---- what a pass cannot do without -------------------------------------------


def work(case):
    m, k = case["rows"], case["width"]
    if case["op"] == "ffn":
        f, b = case["hidden"], _BYTES[case["type"]]
        return {"bytes": b * (m * k + 2 * k * f + m * f * (3 if case["keep"] else 1)), "flops": 4 * m * k * f}
    if case["op"] == "ffn_grad":
        f, b = case["hidden"], _BYTES[case["type"]]
        return {"bytes": b * (2 * m * k + 4 * k * f + m * f * (1 if case["recompute"] else 3)),
                "flops": (12 if case["recompute"] else 8) * m * k * f}
    if case["op"] == "quantize":
        return {"bytes": 2 * m * k * _BYTES[case["type"]], "flops": 4 * m * k}
    n, pair = case["cols"], 1 if case["act"] == "none" else 2
    return {"bytes": m * k * _BYTES[case["type"]] + pair * n * k * 17 / 32 + m * n * _BYTES[case["out"]],
            "flops": 2 * pair * m * n * k}


# ---- the definitions in 64 bits -------------------------------------------------


def exact(case, seed):
    if work(case)["flops"] > 4e12:  # 64-bit products of that size take too long
        return None
    s = prepare(case, seed)
    return {"ffn": _exact_ffn, "ffn_grad": _exact_grad, "quantize": _exact_quantize, "mx_gemm": _exact_gemm}[case["op"]](s)


def _exact_act(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    if kind == "gelu":
        return g * 0.5 * torch.special.erfc(-g / 2**0.5)
    if kind == "gelu_tanh":  # (1 + tanh y) / 2 is the logistic function of 2 y
        return g * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (g + 0.044715 * g**3))
    return g.clamp(min=0) if kind == "relu" else g


def _halves(s):
    """The gate's and the other weights, input by output."""
    w = s["w"].double()
    return (w.t() if s["case"]["linear"] else w).split(s["case"]["hidden"], 1)


def _exact_ffn(s):
    x = s["x"].double()
    wg, wu = _halves(s)
    g, u = x.mm(wg), x.mm(wu)
    out = {"h": _exact_act(g, s["case"]["act"]) * u}
    if s["case"]["keep"]:
        out["preact"] = torch.hstack([g, u])
    return out


def _exact_grad(s):
    case = s["case"]
    x, dh = s["x"].double(), s["dh"].double()
    wg, wu = _halves(s)
    g, u = (x.mm(wg), x.mm(wu)) if case["recompute"] else s["preact"].double().split(case["hidden"], 1)
    leaf = g.detach().clone().requires_grad_()
    with torch.enable_grad():
        a = _exact_act(leaf, case["act"])
        slope, = torch.autograd.grad(a.sum(), leaf)
    dg, du = dh * u * slope, dh * a.detach()
    dw = torch.hstack([x.t().mm(dg), x.t().mm(du)])
    return {"dx": dg.mm(wg.t()) + du.mm(wu.t()), "dw": dw.t() if case["linear"] else dw}


def _power(n):
    return ((n + 1023) << 52).view(torch.float64)


def _nearest(x):
    """Each block's values on the grid of its scale: the nearest, of two equally near the one of even code."""
    rows, width = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -width % 32)).view(rows, -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    # A 64-bit float's own exponent field: the logarithm rounded down.
    power = (top.view(torch.int64) >> 52) - 1023
    scale = _power(power.clamp(-125, 129) - 2)
    grid = torch.tensor([0, 1, 2, 4, 0.5, 1.5, 3, 6], device="cuda", dtype=torch.float64)  # even codes first: they win ties
    best, off = torch.zeros_like(v), torch.full_like(v, math.inf)
    for q in grid.tolist():
        d = (v.abs() / scale - q).abs()
        best, off = torch.where(d < off, q, best), torch.minimum(off, d)
    return (best * scale * v.sign()).view(rows, -1)


def _exact_quantize(s):
    return {"values": _nearest(s["x"])[:, :s["case"]["width"]]}


def _read(s, name):
    """A stored matrix, from its bytes one row tile at a time."""
    codes, scales = s[name + "codes"].long(), s[name + "scales"].long()
    rows, blocks = codes.shape[0], codes.shape[1] // 16
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device="cuda", dtype=torch.float64)
    out = torch.empty(rows, blocks * 32, device="cuda", dtype=torch.float64)
    out[:, 0::2], out[:, 1::2] = table[codes % 16], table[codes // 16]
    r, b = torch.arange(rows, device="cuda")[:, None], torch.arange(blocks, device="cuda")[None]
    e = scales[r // 128, b // 4, r % 32, r % 128 // 32, b % 4]
    return out * _power(e - 127).repeat_interleave(32, 1)


def _exact_gemm(s):
    case = s["case"]
    x = _nearest(s["x"])
    z = x.mm(_read(s, "w_").t()) * case["alpha"]
    if case["act"] != "none":
        z = _exact_act(z, case["act"]) * (x.mm(_read(s, "u_").t()) * case["alpha"])
    return {"out": z}
