"""Temperatures whose square or reciprocal leaves fp32: distributions are one
token's (or the equals'), and the loss, about a logit's difference times the
temperature, keeps its relative accuracy while it is a normal number.

Tolerances: as for large logits. What is below 2^-126 may be lost, and numbers
below it have a spacing of 2^-149, which a few products add up.
"""
import numpy as np
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import lm_reference as ref
from tests.test_distill_gpu import Case as Distill
from tests.test_large_logits_gpu import expected
from tests.test_verify_gpu import NEAR
from tests.test_verify_gpu import Case as Verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


def tau32(tau):
    return float(np.float32(tau))  # what the call has


@pytest.mark.parametrize("tau", [1e-15, 1e-20, 1e-25, 1e-36, 1e-39])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_distillation(dtype, tau):
    for rows, vocab in ((4, 3000), (90, 20000), (4, 50304), (2, 300001)):
        c = Distill(vocab, rows, vocab, 9, dtype, "fp32", tau32(tau))
        c.logits[0, ::7] = 12.0  # equals at the top, some of them the teacher's
        c.logits[1] = 0.0
        loss, lse, d, d2, alone = c.run()
        want, tol, want_lse, grad, grad_tol = expected(c)
        tol = tol + 2.0 ** -126
        ref.assert_within(ref.f64(loss), want, tol, "loss")
        ref.assert_within(ref.f64(alone), want, tol, "loss alone")
        for g, what in ((d, "gradient"), (d2, "gradient from lse")):
            ref.assert_within(ref.f64(g), grad, grad_tol, what)
        assert not lse.isnan().any()


@pytest.mark.parametrize("tau", [1e-20, 1e-36, 1e-39, 1e-44])
@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_verification(dtype, point, tau):
    for vocab in (900, 40000):
        c = Verify(vocab, 10, 3, vocab, dtype, tau32(tau), tau32(tau), point)
        t = c.target.view(10, 4, vocab)
        t[0] = 0.0         # all alike
        t[1, 0, ::5] = 20  # many alike
        c.tokens.copy_(t[:, :3].argmax(-1))
        accepted, out, lp = c.run()
        want = ref.verify(ref.f64(c.target), None if point else ref.f64(c.draft), c.tokens.cpu().numpy(), np.full(10, 3),
                          ref.f64(c.uniforms), ref.f64(c.noise), c.tau, c.draft_tau)
        sure = want[3] > NEAR
        assert sure.sum() >= 8 and (out[np.arange(10), accepted] >= 0).all()
        assert np.array_equal(accepted[sure], want[0][sure]) and np.array_equal(out[sure], want[1][sure])
        ref.assert_within(lp[sure], want[2][sure], 8e-6 + 3e-7 * np.abs(want[2][sure]), "logprobs")
