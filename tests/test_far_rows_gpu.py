"""The gradient of the distillation alone, from a forward call's lse, for rows
far from zero: lse in 32 bits loses of their sum what its spacing is there,
and all of it where logits are a mask's or the type's lowest value.

Tolerances: those of the gradient with its own sums, and beside them for rows
whose lse is taken as it is, with |lse| up to 64 (512 in 16-bit types), what the
rounding of lse, of a logit over the temperature and of lse's own quotient
make of q: 2.5e-7 of |lse|.
"""
import numpy as np
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import lm_reference as ref
from tests.gpu_util import stream
from tests.test_distill_gpu import Case
from tests.test_large_logits_gpu import expected

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


def check(c):
    loss, lse, d, d2, _ = c.run()
    _, _, want_lse, want, tol = expected(c)
    far = 64 if c.dtype == "fp32" else 512
    near = np.where(np.abs(want_lse) <= far * 1.01, np.abs(want_lse), 0.0)[:, None]
    scale = np.abs(ref.f64(c.dloss) * ref.f64(c.weight) * c.tau)[:, None]
    s = ref.f64(c.logits) / c.tau
    ref.assert_within(ref.f64(d), want, tol, "gradient")
    ref.assert_within(ref.f64(d2), want, tol + 2.5e-7 * near * scale * np.exp(ref.log_softmax(s)), "gradient from lse")
    # In the logits' place.
    assert sat.rowop_distill_backward(c.args(lse=lse, dlogits=c.logits, ldd=c.logits.stride(0)), stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(c.logits, d2)


@pytest.mark.parametrize("tau", [1.0, 0.5, 1.5])
@pytest.mark.parametrize("rows,vocab,pad", [(7, 40, 0), (7, 9001, 3), (90, 2000, 0), (7, 50304, 0), (400, 33001, 0), (7, 300001, 3)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_rows_far_from_zero(dtype, rows, vocab, pad, tau):
    c = Case(vocab, rows, vocab, 11, dtype, "fp32", tau, pad, pad)
    low = torch.finfo(ref.TYPES[dtype]).min
    c.logits[0] = low
    c.logits[1] = -6e4 if dtype == "fp16" else -1e10
    c.logits[2] += 5e4 if dtype == "fp16" else 1e6
    c.logits[3] -= 300
    c.logits[4] += 40
    c.weight[5] = 0.0
    check(c)


@pytest.mark.parametrize("tau", [0.2, 0.02, 1e-3])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_low_temperatures(dtype, tau):
    for rows, vocab in ((5, 3000), (5, 70000), (300, 40000)):
        check(Case(rows + vocab, rows, vocab, 20, dtype, "fp32", tau))


def test_rows_without_an_entry():
    c = Case(1, 6, 50000, 4, "bf16")
    c.logits -= 5000
    c.ids[2] = -1
    c.ids[3, 1:] = -1
    _, lse, d, d2, _ = c.run()
    assert bool((d2[2] == 0).all()) and bool((d[2] == 0).all())
    lse[2] = -4e4  # whatever a caller has there
    assert sat.rowop_distill_backward(c.args(lse=lse, dlogits=c.logits, ldd=c.logits.stride(0)), stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(c.logits, d2)
