"""Distillation and verification with finite logits far from zero: masks such
as -1e9, -1e10 or -1e20 in a padded vocabulary's tail, in all but a few tokens
or in whole rows, and temperatures that make ordinary logits large.

Tolerances: the difference of two logits, and its quotient by the temperature,
are good to a few 2^-24 of the difference, so a log-probability is good to
8e-6 + 3e-7 of its own size and a probability to that relatively; gradients
are rounded once more to their type, and what is below the smallest normal
number before the last product may be lost.
"""
import numpy as np
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import lm_reference as ref
from tests.gpu_util import stream
from tests.test_distill_gpu import Case as Distill
from tests.test_verify_gpu import NEAR
from tests.test_verify_gpu import Case as Verify

pytestmark = pytest.mark.gpu

MASKS = [("fp32", -1e9), ("fp32", -1e10), ("fp32", -1e20), ("fp32", -9e29), ("bf16", -1e9), ("bf16", -1e10), ("bf16", -1e20),
         ("bf16", -9e29), ("fp16", -6e4)]
# With every mask, and without one once a type.
MASKED = [(*m, p) for m in MASKS for p in ("none", "tail", "few", "rows") if p != "none" or m[1] in (-1e9, -6e4)]
TAUS = (1.0, 0.1, 1e-5, 1e-9)


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


def size(log_p):
    return 8e-6 + 3e-7 * np.abs(log_p)


def expected(c):
    """(loss, its tolerance, lse, gradient, its tolerance) of a Distill case, in 64 bits."""
    s, t, ids, tau = ref.f64(c.logits), ref.f64(c.teacher), c.ids.cpu().numpy(), c.tau
    weight, dloss = ref.f64(c.weight), ref.f64(c.dloss)
    loss, lse, d, _ = ref.distill(s, ids, t, tau, weight, dloss)
    loss_tol, d_tol = np.zeros_like(loss), np.zeros_like(d)
    for r in range(c.rows):
        log_p, log_q = ref.log_softmax(t[r] / tau), ref.log_softmax(s[r] / tau)
        p, q, at = np.exp(log_p), np.exp(log_q), log_q[ids[r]]
        on = p > 0
        terms = np.abs(log_p - at) * size(log_p) + size(log_p) + size(at)
        loss_tol[r] = abs(weight[r]) * tau ** 2 * (p[on] * terms[on]).sum()
        p_size = (p[on] * size(log_p[on])).sum()
        d_tol[r] = q * np.where(q > 0, size(log_q), 0.0) * p.sum() + q * p_size
        np.add.at(d_tol[r], ids[r][on], (p * size(log_p))[on])
        d_tol[r] = abs(dloss[r] * weight[r] * tau) * (d_tol[r] + 2.0 ** -126)
    return loss, loss_tol + 1e-37, lse, d, d_tol + ref.rounding(c.dtype, d)


def masked(c, low, pattern):
    """Puts `low` into a Distill case's logits, aside from the teacher's tokens unless whole rows are masked."""
    mask = torch.zeros(c.rows, c.vocab, dtype=torch.bool, device="cuda")
    if pattern == "tail":
        mask[:, c.vocab - c.vocab * 3 // 8:] = True
    else:
        mask[:] = True
    if pattern == "few":
        mask[:, 7::c.vocab // 5] = False
    if pattern != "rows":
        mask.scatter_(1, c.ids.long(), False)
    c.logits.masked_fill_(mask, low)


@pytest.mark.parametrize("tau", TAUS)
@pytest.mark.parametrize("dtype,low,pattern", MASKED)
def test_distillation(dtype, low, pattern, tau):
    # A CTA a row of short rows and of many; slices of one row in a CTA and in clusters.
    for rows, vocab in ((3, 5003), (80, 20000), (3, 50304), (2, 300001)):
        c = Distill(rows + vocab, rows, vocab, 9, dtype, "fp32", tau)
        masked(c, low, pattern)
        got_loss, got_lse, d, _, alone = c.run()
        loss, loss_tol, lse, want, tol = expected(c)
        ref.assert_within(ref.f64(got_loss), loss, loss_tol, "loss")
        ref.assert_within(ref.f64(alone), loss, loss_tol, "loss alone")
        over = np.abs(lse) > np.finfo(np.float32).max
        assert np.array_equal(ref.f64(got_lse)[over], np.copysign(np.inf, lse[over]))
        ref.assert_within(ref.f64(got_lse)[~over], lse[~over], size(lse[~over]), "lse")
        ref.assert_within(ref.f64(d), want, tol, "gradient")


def apart(c, b, n, out):
    """Whether sequence b's draw from p - q is beyond what p's rounding (1e-5 of it) at any token may decide."""
    if n == c.drafts:
        return True
    p = np.exp(ref.log_softmax(ref.f64(c.target)[b * (c.drafts + 1) + n] / c.tau))
    r = np.maximum(p - np.exp(ref.log_softmax(ref.f64(c.draft)[b * c.drafts + n] / c.draft_tau)), 0.0)
    e = ref.f64(c.noise)[b]
    return not (r > 0).any() or (r / e)[out[n]] > 1e-5 * (p / e).max()


@pytest.mark.parametrize("mode,tau", [(m, t) for m in ("sampled", "point") for t in TAUS] + [("greedy", 1.0)])
@pytest.mark.parametrize("dtype,low,pattern", MASKED)
def test_verification(dtype, low, pattern, tau, mode):
    batch, drafts = 12, 3
    for vocab in (5003, 40000):
        c = Verify(vocab, batch, drafts, vocab, dtype, 0.0 if mode == "greedy" else tau, tau, mode == "point")
        mask = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        if pattern == "tail":
            mask[vocab - vocab * 3 // 8:] = True
        elif pattern == "few":
            mask[:] = True
            mask[7::vocab // 5] = False
        c.target[:, mask] = low
        if c.draft is not None:
            c.draft[:, mask] = low
        if pattern == "rows":  # every second sequence's first two rows
            c.target.view(batch, drafts + 1, vocab)[::2, :2] = low
        if mode == "greedy":
            c.tokens.copy_(c.target.float().view(batch, drafts + 1, vocab)[:, :drafts].argmax(-1))
            c.tokens[::3, 2] = 1
        accepted, out, lp = c.run()
        # A drafted token of probability 0 on both sides is refused, 0 < 0 being false: no near tie.
        tokens = c.tokens.cpu().numpy()
        if c.draft is not None:
            tokens = np.where(mask.cpu().numpy()[tokens], -1, tokens)
        want = ref.verify(ref.f64(c.target), None if c.draft is None else ref.f64(c.draft), tokens,
                          np.full(batch, drafts), ref.f64(c.uniforms), ref.f64(c.noise), c.tau, c.draft_tau)
        sure = want[3] > NEAR
        if mode == "sampled":
            sure &= [apart(c, b, n, out) for b, (n, out) in enumerate(zip(*want[:2]))]
        # Where a few tokens are left and the temperature puts all mass on one, p and q are often alike.
        assert sure.sum() >= (1 if pattern == "few" else 0.8 * batch) and (out[np.arange(batch), accepted] >= 0).all()
        assert np.array_equal(accepted[sure], want[0][sure]) and np.array_equal(out[sure], want[1][sure])
        ref.assert_within(lp[sure], want[2][sure], size(want[2][sure]), "logprobs")
