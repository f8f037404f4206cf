"""Draft rows without a distribution (nothing allowed, a NaN or +inf in it):
the token is refused, and the next one is drawn from the target's row."""
import numpy as np
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import lm_reference as ref
from tests.test_verify_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab,pad", [(7, 0), (5003, 0), (40000, 3), (131072, 0)])
def test_the_draw_is_from_the_target(dtype, vocab, pad):
    c = Case(3, 8, 3, vocab, dtype, 0.9, pad=pad)
    good = c.run()
    bad = c.draft.view(8, 3, vocab).clone()
    bad[0, 0] = float("-inf")
    bad[1, 0, vocab // 2] = float("nan")
    bad[2, 0, 1] = float("inf")
    bad[3, 0, c.tokens[3, 0]] = float("inf")
    bad[4, 0] = float("nan")
    c.draft.copy_(bad.reshape(24, vocab))
    c.uniforms[:5, 0] = 0.0
    accepted, out, lp = c.run()
    assert (accepted[:5] == 0).all() and (out[:5, 1:] == -1).all()
    log_p = ref.log_softmax(ref.f64(c.target)[0:20:4] / 0.9)
    score = np.exp(log_p) / ref.f64(c.noise)[:5]
    # No near ties among these draws: the winner is ahead by more than fp32 may take away.
    assert (np.sort(score, 1)[:, -2] < 0.9999 * score.max(1)).all()
    assert np.array_equal(out[:5, 0], score.argmax(1))
    ref.assert_within(lp[:5, 0], log_p[np.arange(5), out[:5, 0]], 8e-6 + 3e-7 * np.abs(log_p).max(), "logprobs")
    for a, b in zip((accepted, out, lp), good):
        assert np.array_equal(a[5:], b[5:])
