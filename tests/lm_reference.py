"""Plain 64-bit implementations (numpy) of the row operators of language
models, written from the formulas in include/rowops.h, and what their tests
share: typed device copies with padding around them, and rounding bounds.
"""
import numpy as np
import torch

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# Half the spacing of the type's numbers around 1, and what may be lost below its smallest numbers (in fp32 and bf16,
# and on the way there in fp32, all of what is below the normal ones).
HALF_ULP = {n: (torch.finfo(t).eps / 2, 2.0 ** -25 if n == "fp16" else 2.0 ** -126) for n, t in TYPES.items()}


def rounding(dtype, ref):
    rel, tiny = HALF_ULP[dtype]
    return rel * np.abs(ref) + tiny


def place(x, dtype, pad=0, offset=0, fill=0.0):
    """(view, whole): x on the device in `dtype`, `offset` elements into a buffer with rows `pad` longer, and that buffer."""
    rows, width = x.shape
    whole = torch.full((offset + rows * (width + pad) + 8,), fill, device="cuda", dtype=TYPES[dtype])
    view = whole[offset:offset + rows * (width + pad)].view(rows, width + pad)[:, :width]
    view.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return view, whole


def f64(t):
    return t.double().cpu().numpy()


def sentinel_intact(view, whole, fill):
    """Whether everything of `whole` outside `view` still has the value `fill`."""
    mask = torch.ones_like(whole, dtype=torch.bool)
    at = (view.data_ptr() - whole.data_ptr()) // whole.element_size()
    rows, width = view.shape
    index = at + torch.arange(rows, device="cuda")[:, None] * view.stride(0) + torch.arange(width, device="cuda")[None]
    mask[index.reshape(-1)] = False
    return bool((whole[mask] == fill).all())


def assert_within(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    bad &= ~(np.isnan(ref) & np.isnan(got))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; first at {i}: {got[i]!r} against {ref[i]!r}, "
                             f"tolerance {np.broadcast_to(tol, ref.shape)[i]:.3g}")


# ---- block norm ------------------------------------------------------------------


def norm(v, kind, gamma, beta, eps):
    if kind == "none":
        return v, None, None
    mean = v.mean(1, keepdims=True) if kind == "layer" else np.zeros((v.shape[0], 1))
    r = 1.0 / np.sqrt(((v - mean) ** 2).mean(1, keepdims=True) + eps)
    n = (v - mean) * r
    if gamma is not None:
        n = n * gamma
    if kind == "layer" and beta is not None:
        n = n + beta
    return n, mean, r


def block_norm(x, y, gate, p):
    """p: post, pre, post_gamma, ..., eps, residual_scale, branch_scale. gate: a row for every row, or 1.0."""
    n, pm, pr = norm(y, p["post"], p.get("post_gamma"), p.get("post_beta"), p["eps"])
    h = p["residual_scale"] * x + p["branch_scale"] * gate * n
    z, m, r = norm(h, p["pre"], p.get("pre_gamma"), p.get("pre_beta"), p["eps"])
    return {"n": n, "h": h, "z": z, "post": (pm, pr), "pre": (m, r)}


def norm_backward(v, dn, kind, gamma, mean, r):
    """(dv, dgamma terms, dbeta terms, sizes of dv's summands)."""
    if kind == "none":
        return dn, None, None, np.abs(dn)
    vh = (v - mean) * r
    a = dn if gamma is None else dn * gamma
    s1 = (a * vh).mean(1, keepdims=True)
    s0 = a.mean(1, keepdims=True) if kind == "layer" else 0.0
    size = r * (np.abs(a) + (np.abs(a).mean(1, keepdims=True) if kind == "layer" else 0.0) +
                (np.abs(vh) + np.abs(mean * r)) * np.abs(a * vh).mean(1, keepdims=True))
    return r * (a - s0 - vh * s1), dn * vh, dn, size


def block_norm_backward(y, h, dh, dz, gate, p, post_stats, pre_stats):
    """The gradients, and for each the sum of its summands' sizes; gate gradients per row."""
    out, size = {}, {}
    d, ds = dh, np.abs(dh)
    if p["pre"] != "none":
        back, dg, db, s = norm_backward(h, dz, p["pre"], p.get("pre_gamma"), *pre_stats)
        d, ds = d + back, ds + s
        mean, r = pre_stats
        out["pre_gamma"], size["pre_gamma"] = dg.sum(0), (np.abs(dz) * (np.abs(h) + np.abs(mean)) * r).sum(0)
        out["pre_beta"], size["pre_beta"] = db.sum(0), np.abs(db).sum(0)
    out["dx"], size["dx"] = p["residual_scale"] * d, abs(p["residual_scale"]) * ds
    b, bs = p["branch_scale"] * d, abs(p["branch_scale"]) * ds
    n, ns = y, np.abs(y)
    if p["post"] != "none":
        mean, r = post_stats
        n, ns = (y - mean) * r, (np.abs(y) + np.abs(mean)) * r
        if p.get("post_gamma") is not None:
            n, ns = n * p["post_gamma"], ns * np.abs(p["post_gamma"])
        if p["post"] == "layer" and p.get("post_beta") is not None:
            n, ns = n + p["post_beta"], ns + np.abs(p["post_beta"])
    out["gate"], size["gate"] = b * n, (bs + np.abs(b)) * ns
    dn, dns = b * gate, bs * np.abs(gate)
    dy, dg, db, s = norm_backward(y, dn, p["post"], p.get("post_gamma"), *(post_stats or (None, None)))
    # dn's own rounding reaches dy through the same linear map: its sizes in the place of dn.
    if p["post"] == "none":
        s = dns
    else:
        mean, r = post_stats
        vh, g = np.abs(y - mean) * r + np.abs(mean) * r, 1.0 if p.get("post_gamma") is None else np.abs(p["post_gamma"])
        s = s + r * (dns * g + (dns * g).mean(1, keepdims=True) + vh * (dns * g * vh).mean(1, keepdims=True))
        out["post_gamma"], size["post_gamma"] = dg.sum(0), (dns * vh).sum(0)
        out["post_beta"], size["post_beta"] = db.sum(0), dns.sum(0)
    out["dy"], size["dy"] = dy, s
    return out, size


# ---- distillation -------------------------------------------------------------------


def log_softmax(v, axis=-1):
    m = v.max(axis, keepdims=True)
    d = v - m
    return d - np.log(np.exp(d).sum(axis, keepdims=True))


def distill(s, ids, teacher, tau, weight, dloss, teacher_lse=None):
    """Row by row: loss, lse, dlogits, and the sizes of the loss's summands."""
    rows, vocab = s.shape
    loss, lse, d, size = np.zeros(rows), np.zeros(rows), np.zeros((rows, vocab)), np.zeros(rows)
    for r in range(rows):
        there = [i for i in range(ids.shape[1]) if 0 <= ids[r, i] < vocab and teacher[r, i] != -np.inf]
        if weight[r] == 0 or not there:
            continue
        t = teacher[r, there] / tau
        log_p = t - teacher_lse[r] if teacher_lse is not None else log_softmax(t)
        p = np.exp(log_p)
        log_q = log_softmax(s[r] / tau)
        at = ids[r, there]
        on = p > 0
        loss[r] = weight[r] * tau ** 2 * (p[on] * (log_p[on] - log_q[at][on])).sum()
        size[r] = abs(weight[r]) * tau ** 2 * (p[on] * (1.0 + np.abs(log_p[on]) + np.abs(log_q[at][on]))).sum()
        m = (s[r] / tau).max()
        lse[r] = m + np.log(np.exp(s[r] / tau - m).sum())
        g = np.exp(log_q) * p.sum()
        np.subtract.at(g, at, p)
        d[r] = dloss[r] * weight[r] * tau * g
    return loss, lse, d, size


# ---- verification ---------------------------------------------------------------------


def verify(target, draft, tokens, lengths, uniforms, noise, tau, draft_tau):
    """(accepted, out, logprobs, margins): margins are the relative distances of each sequence's decisions from the
    other outcome, so that what rounding may decide can be told from what it may not."""
    batch, drafts = tokens.shape
    vocab = target.shape[1]
    accepted = np.zeros(batch, int)
    out, lp, margin = -np.ones((batch, drafts + 1), int), np.zeros((batch, drafts + 1)), np.full(batch, np.inf)

    def dist(row, t):
        return np.exp(log_softmax(row / t)) if np.isfinite(row.max()) and not np.isnan(row).any() else None

    for b in range(batch):
        rows = target[b * (drafts + 1):(b + 1) * (drafts + 1)]
        n = 0
        while n < min(max(lengths[b], 0), drafts):
            x, p = tokens[b, n], dist(rows[n], tau or 1.0)
            if p is None or not 0 <= x < vocab:
                break
            if tau == 0:
                if x != rows[n].argmax():
                    break
            else:
                q = 1.0 if draft is None else dist(draft[b * drafts + n], draft_tau)[x]
                margin[b] = min(margin[b], abs(uniforms[b, n] * q - p[x]) / max(p[x], 1e-300))
                if not uniforms[b, n] * q < p[x]:
                    break
            n += 1
        accepted[b] = n
        p = dist(rows[n], tau or 1.0)
        last = -1
        if p is not None and tau == 0:
            last = int(rows[n].argmax())
        elif p is not None:
            r = p
            if n < min(max(lengths[b], 0), drafts):
                x = tokens[b, n]
                if draft is None:
                    r = p.copy()
                    if 0 <= x < vocab:
                        r[x] = 0.0
                else:
                    r = np.maximum(p - dist(draft[b * drafts + n], draft_tau), 0.0)
                if not (r > 0).any():
                    r = p
            score = np.where(r > 0, r / noise[b], -1.0)
            last = int(score.argmax())
            rivals = np.delete(score, last)
            if rivals.size:
                # The size of a difference's rounding is that of p.
                margin[b] = min(margin[b], (score[last] - rivals.max()) / score[last] * r[last] / p[last])
        said = list(tokens[b, :n]) + [last]
        out[b, :n + 1] = said
        for i, x in enumerate(said):
            if x >= 0:
                lp[b, i] = log_softmax(rows[i] / (tau or 1.0))[x]
    return accepted, out, lp, margin
