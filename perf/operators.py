"""The language-model row operators on their real range of sizes: block norm
(the step between two blocks: norm after, gate, residual, norm before),
distillation from a teacher's top logits, and verification of drafted tokens.

``run`` computes them in plain torch operations in 32 bits, or, where ``own``
is true, through the library's entry points. ``exact`` is their definition in
64 bits.
"""
import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
_EPS = 1e-6


def listed():
    norm = {"op": "block_norm", "residual_scale": 1.0, "branch_scale": 1.0, "pad": 0}
    distill = {"op": "distill", "pad": 0}
    verify = {"op": "verify", "pad": 0}
    return [
        # One token of one request passing from a block to the next while decoding.
        {"name": "norm decode 1x4096", **norm, "grad": False, "rows": 1, "width": 4096, "block": "bf16", "stream": "bf16",
         "post": "rms", "pre": "rms", "gate_rows": 1, "gate": "fp32", "stats": False},
        # A long prompt through a wide model, norms before and after the block, no gate.
        {"name": "norm prompt 8192x8192", **norm, "grad": False, "rows": 8192, "width": 8192, "block": "bf16",
         "stream": "bf16", "post": "rms", "pre": "rms", "gate_rows": 0, "gate": "fp32", "stats": False},
        # The forward pass of a training step with an odd width and a padded stride: fp32 throughout, plain
        # pre-norm residual with a learned gate per column, statistics kept for the backward pass.
        {"name": "norm forward 2049x5001 fp32", **norm, "grad": False, "rows": 2049, "width": 5001, "block": "fp32",
         "stream": "fp32", "post": "none", "pre": "layer", "gate_rows": 1, "gate": "fp32", "stats": True, "pad": 3,
         "branch_scale": 0.5},
        # The backward pass of a training step: 16-bit blocks on a 32-bit residual stream.
        {"name": "norm backward 16384x4096", **norm, "grad": True, "rows": 16384, "width": 4096, "block": "bf16",
         "stream": "fp32", "post": "rms", "pre": "rms", "gate_rows": 1, "gate": "fp32", "stats": True},
        # The backward pass with layer norms, one gate row per sequence, an odd width, a scaled residual.
        {"name": "norm backward 4593x1537 layer", **norm, "grad": True, "rows": 4593, "width": 1537, "block": "fp16",
         "stream": "fp16", "post": "layer", "pre": "layer", "gate_rows": 3, "gate": "fp16", "stats": True,
         "residual_scale": 1.25},
        # The last few positions of a micro-batch: loss and gradient in one call.
        {"name": "distill step 7x32000", **distill, "grad": "both", "rows": 7, "vocab": 32000, "k": 20, "type": "bf16",
         "teacher": "fp32", "tau": 2.0, "whole": False, "masked": 0.0},
        # A training step's loss and gradient over a large vocabulary, an eighth of the positions masked (prompts).
        {"name": "distill step 4096x131072", **distill, "grad": "both", "rows": 4096, "vocab": 131072, "k": 64,
         "type": "bf16", "teacher": "bf16", "tau": 1.0, "whole": False, "masked": 0.125},
        # Evaluation: the loss alone, odd vocabulary, the teacher's whole sum known.
        {"name": "distill loss 1000x49999 fp32", **distill, "grad": "none", "rows": 1000, "vocab": 49999, "k": 128,
         "type": "fp32", "teacher": "fp32", "tau": 1.5, "whole": True, "masked": 0.0},
        # The backward pass alone, from the sums that the forward pass kept (an automatic differentiation's call).
        {"name": "distill backward 2047x65537", **distill, "grad": "only", "rows": 2047, "vocab": 65537, "k": 33,
         "type": "fp16", "teacher": "fp16", "tau": 2.0, "whole": False, "masked": 0.0},
        # One request, four drafted tokens: latency counts.
        {"name": "verify 1x4 of 32768", **verify, "batch": 1, "drafts": 4, "vocab": 32768, "type": "bf16", "tau": 1.0,
         "point": False, "ragged": False},
        # A serving batch with a draft model.
        {"name": "verify 64x5 of 131072", **verify, "batch": 64, "drafts": 5, "vocab": 131072, "type": "bf16",
         "tau": 0.8, "point": False, "ragged": True},
        # A large batch with drafts looked up in the text (no draft distribution), odd vocabulary.
        {"name": "verify 193x3 of 65537 point", **verify, "batch": 193, "drafts": 3, "vocab": 65537, "type": "fp16",
         "tau": 1.0, "point": True, "ragged": True},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def capped(n, most):
        return max(1, min(n, most))

    def width(lo, hi):  # half of them multiples of 64, as models have them
        n = size(lo, hi)
        return n if rng.random() < 0.5 else max(64, n // 64 * 64)

    op = rng.choice(["block_norm", "distill", "verify"])
    pad = rng.choice([0, 0, 8, 3])
    if op == "block_norm":
        w = width(64, 16384)
        rows = capped(size(1, 16384), 2**26 // w)
        block = rng.choice(["bf16", "fp16", "fp32"])
        grad = rng.random() < 0.5
        return {"op": op, "grad": grad, "rows": rows, "width": w, "block": block,
                "stream": rng.choice([block, "fp32"]), "post": rng.choice(["none", "rms", "layer"]),
                "pre": rng.choice(["rms", "layer"]), "gate_rows": rng.choice([0, 1, min(rows, 3), rows]),
                "gate": rng.choice([block, "fp32"]), "stats": grad or rng.random() < 0.5, "pad": pad,
                "residual_scale": rng.choice([1.0, 1.25]), "branch_scale": rng.choice([1.0, 0.5])}
    if op == "distill":
        v = width(1000, 262144)
        return {"op": op, "grad": rng.choice(["both", "none", "only"]), "rows": capped(size(1, 4096), 2**28 // v),
                "vocab": v, "k": size(1, 256), "type": rng.choice(["bf16", "fp16", "fp32"]),
                "teacher": rng.choice(["bf16", "fp16", "fp32"]), "tau": rng.choice([1.0, 1.5, 2.0]),
                "whole": rng.random() < 0.3, "masked": rng.choice([0.0, 0.125]), "pad": pad}
    v, drafts = width(1000, 262144), rng.randint(1, 8)
    return {"op": op, "batch": capped(size(1, 256), 2**27 // (v * (2 * drafts + 1))), "drafts": drafts, "vocab": v,
            "type": rng.choice(["bf16", "fp16", "fp32"]), "tau": rng.choice([1.0, 0.8, 0.0]),
            "point": rng.random() < 0.3, "ragged": rng.random() < 0.5, "pad": pad}


# ---- inputs -------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"block_norm": _prepare_norm, "distill": _prepare_distill, "verify": _prepare_verify}[case["op"]](case, g)


def _empty(rows, width, dtype, pad):
    return torch.empty(rows, width + pad, device="cuda", dtype=dtype)[:, :width]


def _randn(g, rows, width, dtype, pad=0, scale=1.0):
    x = _empty(rows, width, dtype, pad)
    x.copy_(torch.randn(rows, width, device="cuda", generator=g) * scale)
    return x


def _stats_of(v, kind):
    """(mean, reciprocal standard deviation or root mean square) of each row, as the forward pass keeps them."""
    if kind == "none":
        return None
    v = v.double()
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    return torch.cat([mean, ((v - mean).square().mean(-1, keepdim=True) + _EPS).rsqrt()], 1).float()


def _prepare_norm(case, g):
    rows, width, pad = case["rows"], case["width"], case["pad"]
    block, stream, gate = _TYPES[case["block"]], _TYPES[case["stream"]], _TYPES[case["gate"]]
    s = {"case": case, "y": _randn(g, rows, width, block, pad, 2.0)}

    def weights(kind, at):
        if kind != "none":
            s[at + "_gamma"] = 1.0 + 0.1 * torch.randn(width, device="cuda", generator=g)
        if kind == "layer":
            s[at + "_beta"] = 0.1 * torch.randn(width, device="cuda", generator=g)

    weights(case["post"], "post")
    weights(case["pre"], "pre")
    s["rows_per_gate"] = -(-rows // case["gate_rows"]) if case["gate_rows"] else rows
    if case["gate_rows"]:
        n = -(-rows // s["rows_per_gate"])
        s["gate"] = (0.5 + 0.2 * torch.randn(n, width, device="cuda", generator=g)).to(gate)
    if case["grad"]:
        s["h"] = _randn(g, rows, width, stream, pad)
        s["dh"] = _randn(g, rows, width, stream, pad)
        s["dz"] = _randn(g, rows, width, block, pad)
        s["post_stats"], s["pre_stats"] = _stats_of(s["y"], case["post"]), _stats_of(s["h"], case["pre"])
        s["dx"], s["dy"] = _empty(rows, width, stream, pad), _empty(rows, width, block, pad)
        for name in ("post_gamma", "post_beta", "pre_gamma", "pre_beta", "gate"):
            if name in s:
                s["d" + name] = torch.empty_like(s[name])
    else:
        s["x"] = _randn(g, rows, width, stream, pad)
        s["h"], s["z"] = _empty(rows, width, stream, pad), _empty(rows, width, block, pad)
        if case["stats"]:
            for at in ("post", "pre"):
                if case[at] != "none":
                    s[at + "_stats"] = torch.empty(rows, 2, device="cuda")
    return s


def _prepare_distill(case, g):
    rows, vocab, k, pad = case["rows"], case["vocab"], case["k"], case["pad"]
    dtype = _TYPES[case["type"]]
    s = {"case": case, "logits": _randn(g, rows, vocab, dtype, pad, 2.5)}
    # The teacher is near the student; its largest logits are what was stored.
    whole = torch.randn(rows, vocab, device="cuda", generator=g).add_(s["logits"], alpha=0.8)
    top, ids = whole.topk(k, dim=-1)
    s["teacher"], s["ids"] = top.to(_TYPES[case["teacher"]]), ids.int()
    if case["whole"]:
        s["teacher_lse"] = (whole / case["tau"]).logsumexp(-1)
    del whole
    # Every fifth row has some entries fewer.
    s["ids"][::5, k - k // 4:] = -1
    s["weight"] = torch.ones(rows, device="cuda")
    s["weight"][torch.randperm(rows, device="cuda", generator=g)[:int(rows * case["masked"])]] = 0.0
    s["loss"], s["lse"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    if case["grad"] != "none":
        # The mean over the rows; in 16-bit floats with the loss scaled up, so that small gradients are not lost.
        s["dloss"] = torch.full((rows,), (4096.0 if case["type"] == "fp16" else 1.0) / rows, device="cuda")
        s["dlogits"] = _empty(rows, vocab, dtype, pad)
    if case["grad"] == "only":
        s["lse"] = (s["logits"].double() / case["tau"]).logsumexp(-1).float()
    return s


def _prepare_verify(case, g):
    batch, drafts, vocab, pad = case["batch"], case["drafts"], case["vocab"], case["pad"]
    dtype = _TYPES[case["type"]]
    s = {"case": case, "target": _randn(g, batch * (drafts + 1), vocab, dtype, pad, 2.5)}
    # The draft model is near the target, and the drafted tokens are its own.
    near = s["target"].float().view(batch, drafts + 1, vocab)[:, :drafts].reshape(batch * drafts, vocab)
    near = near + 0.6 * torch.randn(batch * drafts, vocab, device="cuda", generator=g)
    tau = case["tau"] or 1.0
    noise = torch.empty(batch * drafts, vocab, device="cuda").exponential_(generator=g)
    s["tokens"] = (near / tau - noise.log()).argmax(-1).int().view(batch, drafts)
    if not case["point"]:
        s["draft"] = _empty(batch * drafts, vocab, dtype, pad)
        s["draft"].copy_(near)
    if case["ragged"]:
        s["lengths"] = torch.randint(0, drafts + 1, (batch,), device="cuda", generator=g, dtype=torch.int32)
    s["uniforms"] = torch.rand(batch, drafts, device="cuda", generator=g)
    s["noise"] = _empty(batch, vocab, torch.float32, pad)
    s["noise"].copy_(torch.empty(batch, vocab, device="cuda").exponential_(generator=g).clamp_(min=1e-20))
    s["accepted"] = torch.empty(batch, device="cuda", dtype=torch.int32)
    s["out"] = torch.empty(batch, drafts + 1, device="cuda", dtype=torch.int32)
    s["logprobs"] = torch.empty(batch, drafts + 1, device="cuda")
    return s


# ---- one pass -------------------------------------------------------------------


def run(state):
    case = state["case"]
    if own:
        return _own(state)
    if case["op"] == "block_norm":
        return _plain_norm_grad(state) if case["grad"] else _plain_norm(state)
    return _plain_distill(state) if case["op"] == "distill" else _plain_verify(state)


def _own(s):
    import shape_adaptive_tile_gb300 as sat

    case, stream = s["case"], torch.cuda.current_stream().cuda_stream
    if "call" not in s:  # the argument block that a program keeps beside its buffers
        s["call"] = {"block_norm": _norm_call, "distill": _distill_call, "verify": _verify_call}[case["op"]](sat, s)
    if case["op"] == "block_norm":
        if case["grad"]:
            sat.check(sat.rowop_block_norm_backward(*s["call"], stream))
            return _norm_grads(s)
        sat.check(sat.rowop_block_norm(*s["call"], stream))
        return {n: s[n] for n in ("h", "z", "post_stats", "pre_stats") if n in s}
    if case["op"] == "distill":
        if case["grad"] == "only":
            sat.check(sat.rowop_distill_backward(s["call"], stream))
            return {"dlogits": s["dlogits"]}
        sat.check(sat.rowop_distill(s["call"], stream))
        return {n: s[n] for n in ("loss", "lse", "dlogits") if n in s}
    sat.check(sat.rowop_verify(s["call"], stream))
    return {n: s[n] for n in ("accepted", "out", "logprobs")}


def _norm_call(sat, s):
    case = s["case"]
    args = sat.BlockNormArgs(
        rows=case["rows"], width=case["width"], block_type=case["block"], stream_type=case["stream"],
        gate_type=case["gate"], post_norm=case["post"], pre_norm=case["pre"], post_eps=_EPS, pre_eps=_EPS,
        residual_scale=case["residual_scale"], branch_scale=case["branch_scale"],
        x=s.get("x"), ldx=s["x"].stride(0) if "x" in s else 0, y=s["y"], ldy=s["y"].stride(0),
        post_gamma=s.get("post_gamma"), post_beta=s.get("post_beta"), pre_gamma=s.get("pre_gamma"),
        pre_beta=s.get("pre_beta"), gate=s.get("gate"), ldg=case["width"], rows_per_gate=s["rows_per_gate"],
        h=s["h"], ldh=s["h"].stride(0), z=s.get("z"), ldz=s["z"].stride(0) if "z" in s else 0,
        post_stats=s.get("post_stats"), pre_stats=s.get("pre_stats"))
    if not case["grad"]:
        return (args,)
    size = sat.rowop_block_norm_workspace(args)
    s["workspace"] = torch.empty(max(1, size), device="cuda", dtype=torch.uint8)
    return args, sat.BlockNormGrads(
        dh=s["dh"], lddh=s["dh"].stride(0), dz=s["dz"], lddz=s["dz"].stride(0), dx=s["dx"], lddx=s["dx"].stride(0),
        dy=s["dy"], lddy=s["dy"].stride(0), dgate=s.get("dgate"), lddg=case["width"],
        dpost_gamma=s.get("dpost_gamma"), dpost_beta=s.get("dpost_beta"), dpre_gamma=s.get("dpre_gamma"),
        dpre_beta=s.get("dpre_beta"), workspace=s["workspace"], workspace_bytes=size)


def _distill_call(sat, s):
    case = s["case"]
    return sat.DistillArgs(
        rows=case["rows"], vocab=case["vocab"], k=case["k"], logits_type=case["type"], teacher_type=case["teacher"],
        temperature=case["tau"], logits=s["logits"], ldl=s["logits"].stride(0), ids=s["ids"], ldi=case["k"],
        teacher=s["teacher"], ldt=case["k"], teacher_lse=s.get("teacher_lse"), weight=s["weight"], loss=s["loss"],
        lse=s["lse"], dloss=s.get("dloss"), dlogits=s.get("dlogits"),
        ldd=s["dlogits"].stride(0) if "dlogits" in s else 0)


def _verify_call(sat, s):
    case = s["case"]
    size = sat.rowop_verify_workspace(case["batch"], case["drafts"], case["vocab"])
    s["workspace"] = torch.empty(max(1, size), device="cuda", dtype=torch.uint8)
    return sat.VerifyArgs(
        batch=case["batch"], drafts=case["drafts"], vocab=case["vocab"], logits_type=case["type"],
        temperature=case["tau"], draft_temperature=case["tau"] or 1.0, target=s["target"],
        ldt=s["target"].stride(0), draft=s.get("draft"), ldq=s["draft"].stride(0) if "draft" in s else 0,
        tokens=s["tokens"], lengths=s.get("lengths"), uniforms=s["uniforms"], noise=s["noise"],
        ldn=s["noise"].stride(0), accepted=s["accepted"], out=s["out"], logprobs=s["logprobs"],
        workspace=s["workspace"], workspace_bytes=size)


def _norm_grads(s):
    names = ("dx", "dy", "dgate", "dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta")
    return {n: s[n] for n in names if n in s}


def _norm(v, kind, gamma, beta):
    """(normed, mean, reciprocal deviation) of the rows of v."""
    if kind == "none":
        return v, None, None
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    r = 1.0 / torch.sqrt((v - mean).square().mean(-1, keepdim=True) + _EPS)
    n = (v - mean) * r * gamma
    return (n + beta if kind == "layer" else n), mean, r


def _gate_rows(s):
    """The gate's row for every row, in 32 bits."""
    rows = s["case"]["rows"]
    return s["gate"].float()[torch.arange(rows, device="cuda") // s["rows_per_gate"]]


def _plain_norm(s):
    case = s["case"]
    n, pm, pr = _norm(s["y"].float(), case["post"], s.get("post_gamma"), s.get("post_beta"))
    if "gate" in s:
        n = n * _gate_rows(s)
    h = case["residual_scale"] * s["x"].float() + case["branch_scale"] * n
    z, m, r = _norm(h, case["pre"], s.get("pre_gamma"), s.get("pre_beta"))
    s["h"].copy_(h)
    s["z"].copy_(z)
    out = {"h": s["h"], "z": s["z"]}
    if case["stats"]:
        if pr is not None:
            out["post_stats"] = torch.cat([pm, pr], 1)
        if r is not None:
            out["pre_stats"] = torch.cat([m, r], 1)
    return out


def _norm_back(v, stats, dn, kind, gamma):
    """Of a norm of the rows of v whose output's gradient is dn: (gradient of v, of gamma, of beta, the normed rows)."""
    if kind == "none":
        return dn, None, None, v
    mean, r = stats[:, :1], stats[:, 1:]
    vh = (v - mean) * r
    a = dn * gamma
    off = (a * vh).mean(-1, keepdim=True) * vh
    if kind == "layer":
        off = off + a.mean(-1, keepdim=True)
    return r * (a - off), (dn * vh).sum(0), dn.sum(0), vh


def _plain_norm_grad(s):
    case = s["case"]
    back, dg, db, _ = _norm_back(s["h"].float(), s["pre_stats"], s["dz"].float(), case["pre"], s.get("pre_gamma"))
    dh = s["dh"].float() + back
    out = {"dx": s["dx"], "dy": s["dy"], "dpre_gamma": dg}
    if case["pre"] == "layer":
        out["dpre_beta"] = db
    s["dx"].copy_(case["residual_scale"] * dh)
    b = case["branch_scale"] * dh
    dn = b * _gate_rows(s) if "gate" in s else b
    dy, dg, db, yh = _norm_back(s["y"].float(), s["post_stats"], dn, case["post"], s.get("post_gamma"))
    s["dy"].copy_(dy)
    if case["post"] != "none":
        out["dpost_gamma"] = dg
    if case["post"] == "layer":
        out["dpost_beta"] = db
    if "gate" in s:
        n = yh if case["post"] == "none" else yh * s["post_gamma"]
        if case["post"] == "layer":
            n = n + s["post_beta"]
        per = torch.zeros(s["gate"].shape, device="cuda")
        if s["gate"].shape[0] == 1:
            per[0] = (b * n).sum(0)
        else:
            per.index_add_(0, torch.arange(case["rows"], device="cuda") // s["rows_per_gate"], b * n)
        out["dgate"] = per.to(s["gate"].dtype)
    return {n: out[n] for n in _norm_grads({**s, **out}) if n in out}


def _plain_distill(s):
    case = s["case"]
    tau, ids = case["tau"], s["ids"].long()
    l = s["logits"].float() / tau
    if case["grad"] == "only":
        lse = s["lse"][:, None]
    else:
        m = l.amax(-1, keepdim=True)
        lse = m + (l - m).exp().sum(-1, keepdim=True).log()
    t = torch.where(ids >= 0, s["teacher"].float() / tau, -math.inf)
    if case["whole"]:
        logp = t - s["teacher_lse"][:, None]
    else:
        m = t.amax(-1, keepdim=True)
        logp = t - (m + (t - m).exp().sum(-1, keepdim=True).log())
    p = logp.exp()
    on = s["weight"][:, None] != 0
    scale = torch.where(on, s["weight"][:, None], 0.0)
    out = {}
    if case["grad"] != "only":
        logq = l.gather(1, ids.clamp(min=0)) - lse
        kl = torch.where(p > 0, p * (logp - logq), 0.0).sum(-1, keepdim=True)
        out["loss"] = torch.where(on, scale * tau * tau * kl, 0.0)[:, 0]
        out["lse"] = torch.where(on, lse, 0.0)[:, 0]
    if case["grad"] != "none":
        d = (l - lse).exp() * p.sum(-1, keepdim=True)
        d.scatter_add_(1, ids.clamp(min=0), -p)
        s["dlogits"].copy_(torch.where(on, d * (scale * tau * s["dloss"][:, None]), 0.0))
        out["dlogits"] = s["dlogits"]
    return out


def _first_of_largest(v):
    at = torch.arange(v.shape[-1], device=v.device)
    return torch.where(v == v.amax(-1, keepdim=True), at, v.shape[-1]).amin(-1)


def _log_probs(x, tau):
    x = x.float() / tau
    x = x - x.amax(-1, keepdim=True)
    return x - x.exp().sum(-1, keepdim=True).log()


def _plain_verify(s):
    case = s["case"]
    batch, drafts, vocab = case["batch"], case["drafts"], case["vocab"]
    tokens, at = s["tokens"].long(), torch.arange(batch, device="cuda")
    logp = _log_probs(s["target"], case["tau"] or 1.0).view(batch, drafts + 1, vocab)
    lengths = s["lengths"].long() if "lengths" in s else torch.full((batch,), drafts, device="cuda")
    inside = torch.arange(drafts, device="cuda") < lengths[:, None]
    said = logp[:, :drafts].gather(2, tokens[:, :, None])[:, :, 0]
    if case["tau"] == 0:
        best = _first_of_largest(s["target"].float()).view(batch, drafts + 1)
        n = ((tokens == best[:, :drafts]) & inside).long().cumprod(1).sum(1)
        token = best[at, n]
    else:
        if case["point"]:
            q = torch.ones_like(said)
        else:
            logq = _log_probs(s["draft"], case["tau"]).view(batch, drafts, vocab)
            q = logq.gather(2, tokens[:, :, None])[:, :, 0].exp()
        n = ((s["uniforms"] * q < said.exp()) & inside).long().cumprod(1).sum(1)
        p, last = logp[at, n].exp(), n.clamp(max=drafts - 1)
        if case["point"]:
            q = torch.zeros_like(p).scatter_(1, tokens[at, last][:, None], 2.0)
        else:
            q = logq[at, last].exp()
        r = torch.where((n < lengths)[:, None], (p - q).clamp(min=0), p)
        r = torch.where((r > 0).any(1, keepdim=True), r, p)
        token = _first_of_largest(r / s["noise"])
    where = torch.arange(drafts + 1, device="cuda")
    padded = torch.cat([tokens, tokens[:, :1]], 1)
    out = torch.where(where < n[:, None], padded, torch.where(where == n[:, None], token[:, None], -1))
    lp = torch.where(out >= 0, logp.gather(2, out.clamp(min=0)[:, :, None])[:, :, 0], 0.0)
    return {"accepted": n.int(), "out": out.int(), "logprobs": lp}


# ---- what a pass cannot do without -------------------------------------------


def work(case):
    if case["op"] == "block_norm":
        n, w = case["rows"] * case["width"], case["width"]
        b, st = _BYTES[case["block"]], _BYTES[case["stream"]]
        vectors = (case["post"] != "none") + (case["post"] == "layer") + (case["pre"] != "none") + (case["pre"] == "layer")
        gate = -(-case["rows"] // -(-case["rows"] // case["gate_rows"])) * w * _BYTES[case["gate"]] if case["gate_rows"] else 0
        stats = 8 * case["rows"] * ((case["post"] != "none") + (case["pre"] != "none")) if case["stats"] else 0
        if case["grad"]:  # reads dh, h, dz, y and writes dx, dy; the weights and the gate read, their gradients written
            return {"bytes": n * 3 * (b + st) + 2 * (vectors * 4 * w + gate) + stats, "flops": 30 * n}
        return {"bytes": n * 2 * (b + st) + vectors * 4 * w + gate + stats, "flops": 14 * n}
    if case["op"] == "distill":
        rows = case["rows"] - int(case["rows"] * case["masked"])
        small = rows * case["k"] * (4 + _BYTES[case["teacher"]]) + case["rows"] * 16
        b = _BYTES[case["type"]] * case["vocab"]
        written = case["rows"] * b if case["grad"] != "none" else 0
        return {"bytes": rows * b + written + small, "flops": (8 if case["grad"] == "both" else 4) * rows * case["vocab"]}
    # All rows of the drafted lengths (on average half of them where they are ragged): nothing says beforehand
    # which of them an early refusal makes needless. One row of noise per sequence.
    d = case["drafts"] * (0.5 if case["ragged"] else 1.0)
    rows = d + 1 + (0 if case["point"] or case["tau"] == 0 else d)
    noise = 4 if case["tau"] else 0
    return {"bytes": case["batch"] * case["vocab"] * (rows * _BYTES[case["type"]] + noise),
            "flops": 4 * case["batch"] * case["vocab"] * rows}


# ---- the definitions in 64 bits -------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "block_norm":
        return _exact_norm_grad(s) if case["grad"] else _exact_norm(s)
    return _exact_distill(s) if case["op"] == "distill" else _exact_verify(s)


def _f64(s, name, default=0.0):
    return s[name].double() if s.get(name) is not None else torch.full((1, 1), default, device="cuda", dtype=torch.float64)


def _moments(v, kind):
    mu = v.sum(1, keepdim=True) / v.shape[1] if kind == "layer" else torch.zeros(v.shape[0], 1, device="cuda").double()
    var = ((v - mu) ** 2).sum(1, keepdim=True) / v.shape[1]
    return mu, (var + _EPS) ** -0.5


def _every_row(s):
    g = _f64(s, "gate", 1.0)
    return g.repeat_interleave(s["rows_per_gate"], 0)[:s["case"]["rows"]] if "gate" in s else g


def _exact_norm(s):
    case = s["case"]
    y, stats = s["y"].double(), {}
    if case["post"] != "none":
        mu, r = _moments(y, case["post"])
        stats["post_stats"] = torch.hstack([mu, r])
        y = _f64(s, "post_gamma") * ((y - mu) * r) + _f64(s, "post_beta")
    h = s["x"].double() * case["residual_scale"] + y * _every_row(s) * case["branch_scale"]
    mu, r = _moments(h, case["pre"])
    stats["pre_stats"] = torch.hstack([mu, r])
    z = _f64(s, "pre_gamma") * ((h - mu) * r) + _f64(s, "pre_beta")
    return {"h": h, "z": z, **(stats if case["stats"] else {})}


def _exact_norm_grad(s):
    """Vector-Jacobian products of the forward formulas, row by row: for v -> (v - mu) r with weights, the
    Jacobian's transpose is r (I - ones/width [layer] - vh vh'/width)."""
    case, width, out = s["case"], s["case"]["width"], {}
    h, y, dz, dh = s["h"].double(), s["y"].double(), s["dz"].double(), s["dh"].double()
    mu, r = _moments(h, case["pre"])
    hh = (h - mu) * r
    up = dz * _f64(s, "pre_gamma")
    down = up - hh * ((up * hh).sum(1, keepdim=True) / width)
    if case["pre"] == "layer":
        down = down - up.sum(1, keepdim=True) / width
        out["dpre_beta"] = dz.sum(0)
    out["dpre_gamma"] = (dz * hh).sum(0)
    total = dh + r * down
    out["dx"] = total * case["residual_scale"]
    total = total * case["branch_scale"]
    gate = _every_row(s)
    if case["post"] == "none":
        n, out["dy"] = y, total * gate
    else:
        mu, r = _moments(y, case["post"])
        yh = (y - mu) * r
        n = yh * _f64(s, "post_gamma") + _f64(s, "post_beta")
        out["dpost_gamma"] = (total * gate * yh).sum(0)
        up = total * gate * _f64(s, "post_gamma")
        down = up - yh * ((up * yh).sum(1, keepdim=True) / width)
        if case["post"] == "layer":
            down = down - up.sum(1, keepdim=True) / width
            out["dpost_beta"] = (total * gate).sum(0)
        out["dy"] = r * down
    if "gate" in s:
        per, short = s["rows_per_gate"], s["gate"].shape[0] * s["rows_per_gate"] - case["rows"]
        v = torch.cat([total * n, torch.zeros(short, width, device="cuda", dtype=torch.float64)])
        out["dgate"] = v.view(-1, per, width).sum(1)
    return out


def _exact_distill(s):
    case = s["case"]
    tau, w = case["tau"], s["weight"].double()[:, None]
    l = s["logits"].double() / tau
    lse = torch.logsumexp(l, 1, keepdim=True)
    there = s["ids"] >= 0
    ids = torch.where(there, s["ids"], 0).long()
    t = (s["teacher"].double() / tau).masked_fill(~there, -math.inf)
    logp = t - (s["teacher_lse"].double()[:, None] if case["whole"] else torch.logsumexp(t, 1, keepdim=True))
    p, out = logp.exp(), {}
    if case["grad"] != "only":
        terms = (p * (logp - l.gather(1, ids) + lse)).masked_fill(p == 0, 0.0)
        out["loss"] = (w * tau ** 2 * terms.sum(1, keepdim=True))[:, 0]
        out["lse"] = (lse * (w != 0))[:, 0]
    if case["grad"] != "none":
        d = l.sub_(lse).exp_().mul_(p.sum(1, keepdim=True))
        d.scatter_add_(1, ids, -p)
        out["dlogits"] = d.mul_(w * tau * s["dloss"].double()[:, None])
    return out


def _exact_verify(s):
    case = s["case"]
    batch, drafts, vocab, tau = case["batch"], case["drafts"], case["vocab"], case["tau"]
    logp = torch.log_softmax(s["target"].double() / (tau or 1.0), 1).view(batch, drafts + 1, vocab)
    logq = torch.log_softmax(s["draft"].double() / (tau or 1.0), 1).view(batch, drafts, vocab) if "draft" in s else None
    accepted, out, lps = [], [], []
    tokens, uniforms = s["tokens"].tolist(), s["uniforms"].tolist()
    lengths = s["lengths"].tolist() if "lengths" in s else [drafts] * batch
    greedy = None
    if not tau:  # the first of the largest
        greedy = [[int((r == r.max()).nonzero()[0]) for r in rows] for rows in logp]
    for b in range(batch):
        n = 0
        while n < lengths[b]:
            x = tokens[b][n]
            if greedy:
                ok = x == greedy[b][n]
            else:
                ok = uniforms[b][n] * (1.0 if logq is None else float(logq[b, n, x].exp())) < float(logp[b, n, x].exp())
            if not ok:
                break
            n += 1
        if greedy:
            last = greedy[b][n]
        else:
            r = logp[b, n].exp()
            if n < lengths[b]:
                if logq is None:
                    r[tokens[b][n]] = 0.0
                else:
                    r = (r - logq[b, n].exp()).clamp(min=0)
                if not bool((r > 0).any()):
                    r = logp[b, n].exp()
            last = int((r / s["noise"][b].double()).argmax())
        said = tokens[b][:n] + [last]
        accepted.append(n)
        out.append(said + [-1] * (drafts - n))
        lps.append([float(logp[b, i, x]) for i, x in enumerate(said)] + [0.0] * (drafts - n))
    return {"accepted": torch.tensor(accepted, dtype=torch.int32), "out": torch.tensor(out, dtype=torch.int32),
            "logprobs": torch.tensor(lps, dtype=torch.float64)}
