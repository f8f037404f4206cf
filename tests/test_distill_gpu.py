"""Distillation from a teacher's top logits against the formulas in 64 bits.

Tolerances: a difference of two logits over the temperature is exact to a few
2^-24 of the logits' range R, and an exponential or logarithm adds about 2^-22;
sums over a row have up to 600 sequential additions in a thread, all of one
sign, at most 600 x 2^-24 / 2 = 2e-5 and, as roundings do not line up, about
1e-6. So probabilities are good to 8e-6 + 3e-7 R relatively, log-probabilities
to that absolutely, and gradients are rounded once more to their type.
"""
import numpy as np
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import lm_reference as ref
from tests.gpu_util import stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


class Case:
    def __init__(self, seed, rows, vocab, k, dtype="fp32", teacher="fp32", tau=1.0, pad=0, offset=0, whole=False, spread=2.5,
                 dloss=None):
        rng = np.random.default_rng(seed)
        self.rows, self.vocab, self.k, self.dtype, self.tau = rows, vocab, k, dtype, tau
        self.pad, self.offset, self.teacher_type = pad, offset, teacher
        self.logits, _ = ref.place(rng.standard_normal((rows, vocab)) * spread, dtype, pad, offset)
        ids = np.stack([rng.permutation(vocab)[:k] if k <= vocab else rng.integers(0, vocab, k) for _ in range(rows)])
        self.ids = torch.from_numpy(ids.reshape(rows, k).astype(np.int32)).cuda()
        self.teacher, _ = ref.place(-np.sort(rng.standard_normal((rows, k)) * 3), teacher, pad, offset)
        self.weight = torch.from_numpy(rng.uniform(0.5, 2.0, rows)).float().cuda()
        self.dloss = torch.from_numpy(rng.standard_normal(rows) if dloss is None else np.full(rows, dloss)).float().cuda()
        self.teacher_lse = None
        if whole:
            t = ref.f64(self.teacher) / tau
            self.teacher_lse = torch.from_numpy(np.log(np.exp(t).sum(1) + rng.uniform(1, 5, rows))).float().cuda()

    def args(self, **more):
        f = dict(rows=self.rows, vocab=self.vocab, k=self.k, logits_type=self.dtype, teacher_type=self.teacher_type,
                 temperature=self.tau, logits=self.logits, ldl=self.logits.stride(0), ids=self.ids, ldi=max(self.k, 1),
                 teacher=self.teacher, ldt=self.teacher.stride(0), teacher_lse=self.teacher_lse, weight=self.weight,
                 dloss=self.dloss)
        return sat.DistillArgs(**{**f, **more})

    def run(self):
        """(loss, lse, gradient of one call, gradient of the backward call), NaN wherever nothing was written."""
        loss, lse = (torch.full((self.rows,), float("nan"), device="cuda") for _ in range(2))
        ds, wholes = zip(*(ref.place(np.full((self.rows, self.vocab), np.nan), self.dtype, self.pad, self.offset, -77.0)
                           for _ in range(2)))
        assert sat.rowop_distill(self.args(loss=loss, lse=lse, dlogits=ds[0], ldd=ds[0].stride(0)), stream()) == 0, \
            sat.gemm_last_error()
        assert sat.rowop_distill_backward(self.args(lse=lse, dlogits=ds[1], ldd=ds[1].stride(0)), stream()) == 0, \
            sat.gemm_last_error()
        alone = torch.full((self.rows,), float("nan"), device="cuda")
        assert sat.rowop_distill(self.args(loss=alone), stream()) == 0, sat.gemm_last_error()
        torch.cuda.synchronize()
        for d, w in zip(ds, wholes):
            assert ref.sentinel_intact(d, w, -77.0)
        return loss, lse, ds[0], ds[1], alone

    def check(self):
        loss, lse, d, d2, alone = self.run()
        s, t, tau = ref.f64(self.logits), ref.f64(self.teacher), self.tau
        weight, dloss = ref.f64(self.weight), ref.f64(self.dloss)
        good = ref.distill(s, self.ids.cpu().numpy(), t, tau, weight, dloss,
                           None if self.teacher_lse is None else ref.f64(self.teacher_lse))
        finite = np.where(np.isfinite(s) & (np.abs(s) < 1e30), s, 0.0)
        span = (finite.max(1) - finite.min(1) + (np.ptp(np.where(np.isfinite(t), t, 0.0), 1) if self.k else 0)) / tau
        rel = 8e-6 + 3e-7 * span
        far = 3e-7 * np.abs(finite).max(1) / tau
        ref.assert_within(ref.f64(loss), good[0], rel * good[3] + 1e-12, "loss")
        ref.assert_within(ref.f64(alone), good[0], rel * good[3] + 1e-12, "loss alone")
        ref.assert_within(ref.f64(lse), good[1], rel + far, "lse")
        q = np.zeros_like(s)
        on = (good[1] != 0) | (good[0] != 0)
        q[on] = np.exp(ref.log_softmax(s[on] / tau))
        p_sum = np.zeros_like(s)
        for r in range(self.rows):
            there = (ref.f64(self.ids[r]) >= 0) & (ref.f64(self.ids[r]) < self.vocab) & (t[r] != -np.inf)
            i = self.ids[r].cpu().numpy()[there]
            lt = t[r, there] / tau
            p = np.exp(lt - (ref.f64(self.teacher_lse)[r] if self.teacher_lse is not None else
                             lt.max() + np.log(np.exp(lt - lt.max()).sum()))) if len(i) else lt
            np.add.at(p_sum[r], i, p)
        size = np.abs(dloss * weight * tau)[:, None] * (q * p_sum.sum(1, keepdims=True) + p_sum)
        # The backward call starts from lse in 32 bits: an absolute error of that, relative in q.
        for got, more, what in ((d, 0.0, "gradient"), (d2, far[:, None], "gradient from lse")):
            ref.assert_within(ref.f64(got), good[2], (rel[:, None] + more) * size + ref.rounding(self.dtype, good[2]), what)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (2, 2, 1), (3, 31, 5), (5, 1000, 20), (2, 4096, 64), (7, 32000, 20),
                                          (3, 49999, 128), (2, 65537, 33), (2, 131072, 64), (1, 262144, 1024),
                                          (1, 300001, 3), (40, 513, 100), (700, 257, 8)])
def test_sizes_and_types(rows, vocab, k, dtype):
    Case(vocab + k, rows, vocab, k, dtype, ("fp32", "bf16", "fp16")[k % 3], (1.0, 2.0, 0.7)[rows % 3]).check()


@pytest.mark.parametrize("i", range(40))
def test_random_strides_and_offsets(i):
    rng = np.random.default_rng(i)
    vocab = int(2 ** rng.uniform(0, 16.5))
    Case(i, int(rng.integers(1, 1 + min(64, 600000 // vocab))), vocab, int(rng.integers(1, min(vocab, 300) + 1)),
         ("fp32", "bf16", "fp16")[i % 3], ("fp32", "bf16", "fp16")[i // 3 % 3], float(rng.choice([0.5, 1.0, 3.0])),
         int(rng.choice([0, 1, 3, 8])), int(rng.choice([0, 1, 5, 8])), bool(i % 2)).check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab,k,pad", [(40, 7, 0), (9001, 300, 0), (16384, 5, 8), (16400, 33, 0), (33001, 12, 3)])
def test_many_rows(vocab, k, pad, dtype):
    # More rows than two an SM: a CTA each, of short rows and of long ones; in place too.
    c = Case(vocab, 306, vocab, min(k, vocab), dtype, "fp32", 1.5, pad, pad)
    c.weight[::7] = 0.0
    c.ids[5] = -1
    c.check()
    loss, lse, d, d2, _ = c.run()
    assert sat.rowop_distill(c.args(loss=lse, dlogits=c.logits, ldd=c.logits.stride(0)), stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(c.logits, d) and torch.equal(loss, lse)


@pytest.mark.parametrize("vocab", [50, 5000, 70000, 280000])
def test_gradient_rows_on_other_bytes_than_the_logits(vocab):
    for rows in (5, 306 if vocab < 10000 else 6):
        c = Case(4, rows, vocab, 9, "bf16")
        loss, lse, d, _, _ = c.run()
        e, whole = ref.place(np.zeros((rows, vocab)), "bf16", 1, 3, -77.0)
        assert sat.rowop_distill(c.args(loss=loss, dlogits=e, ldd=e.stride(0)), stream()) == 0
        torch.cuda.synchronize()
        assert torch.equal(d, e) and ref.sentinel_intact(e, whole, -77.0)


@pytest.mark.parametrize("vocab", [50, 5000, 70000, 280000])
def test_masked_and_absent(vocab):
    c = Case(4, 9, vocab, 24, "bf16", "bf16", 2.0)
    c.weight[2] = 0.0
    c.logits[2] = float("nan")  # not read
    c.ids[3] = -1               # no entry at all
    c.logits[3, 1] = float("inf")
    c.teacher[4] = float("-inf")
    c.ids[5, 10:] = -1
    c.teacher[5, 10:] = float("nan")  # of absent entries
    c.ids[6, 3] = vocab               # outside the vocabulary
    c.ids[6, 4] = 2 ** 31 - 1
    c.teacher[7, 5:] = float("-inf")
    loss, lse, d, d2, _ = c.run()
    for r in (2, 3, 4):
        assert loss[r] == 0 and lse[r] == 0 and bool((d[r] == 0).all()) and bool((d2[r] == 0).all())
    c.logits[2:4] = 0.0
    c.teacher[5, 10:] = 0.0
    c.check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [64, 33000, 140000])
def test_infinite_and_lowest_student_logits(dtype, vocab):
    c = Case(6, 5, vocab, 10, dtype, "fp32", 1.5)
    low = torch.finfo(ref.TYPES[dtype]).min
    outside = torch.ones(5, vocab, dtype=torch.bool, device="cuda")
    outside.scatter_(1, c.ids.long(), False)
    c.logits[0, outside[0]] = float("-inf")  # only the teacher's tokens are allowed
    c.logits[1, outside[1]] = low
    c.logits[2] = low                        # all equal: uniform
    c.logits[3, vocab // 2:] = torch.where(outside[3, vocab // 2:], float("-inf"), c.logits[3, vocab // 2:])
    c.logits[4] += 10000 if dtype != "fp16" else 1000
    loss, lse, d, d2, _ = c.run()
    # Row 2's logits are past what the bounds below are made for: its distribution is uniform.
    want = np.full(vocab, 1.0 / vocab)
    t = ref.f64(c.teacher[2]) / 1.5
    np.subtract.at(want, c.ids[2].cpu().numpy(), np.exp(ref.log_softmax(t)))
    want *= float(c.dloss[2]) * float(c.weight[2]) * 1.5
    ref.assert_within(ref.f64(d[2]), want, 2e-5 * np.abs(want) + 1e-6 / vocab + ref.rounding(dtype, want), "uniform row")
    c.logits[2] = 0.0
    c.check()


def test_the_highest_student_logit_alone():
    # All mass on one token, the teacher's second: log q of the others is far below.
    c = Case(6, 2, 1000, 2, "fp32", "fp32", 1.0)
    c.logits[:] = 0.0
    c.logits[:, 7] = 200.0
    c.ids[:] = torch.tensor([3, 7])
    c.check()


def test_repeated_ids_add_up():
    c = Case(9, 4, 3000, 6, "fp32", "fp32", 1.0)
    c.ids[0] = torch.tensor([5, 5, 5, 5, 5, 5])
    c.ids[1] = torch.tensor([5, 6, 5, 6, 7, 5])
    c.ids[2] = torch.tensor([2999, 0, 2999, 0, -1, -1])
    c.check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab,pad", [(40, 0), (5003, 0), (40000, 8), (150001, 3), (262144, 0)])
def test_gradient_in_place_and_repeats(vocab, pad, dtype):
    c = Case(5, 6, vocab, 30, dtype, "fp32", 1.0, pad)
    loss, lse, d, d2, _ = c.run()
    loss2, lse2, e, e2, _ = c.run()
    assert all(torch.equal(a, b) for a, b in ((loss, loss2), (lse, lse2), (d, e), (d2, e2)))
    keep = c.logits.clone()
    assert sat.rowop_distill(c.args(loss=loss2, lse=lse2, dlogits=c.logits, ldd=c.logits.stride(0)), stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(c.logits, d) and torch.equal(loss, loss2)
    c.logits.copy_(keep)
    assert sat.rowop_distill_backward(c.args(lse=lse, dlogits=c.logits, ldd=c.logits.stride(0)), stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(c.logits, d2)


def test_no_entries_and_defaults():
    c = Case(1, 3, 100, 1, "fp32")
    loss, lse, d, _, _ = c.run()
    got = torch.full((3,), float("nan"), device="cuda")
    dn = torch.full((3, 100), float("nan"), device="cuda")
    assert sat.rowop_distill(sat.DistillArgs(rows=3, vocab=100, k=0, temperature=1.0, logits=c.logits, ldl=c.logits.stride(0),
                                             loss=got, dlogits=dn, ldd=100), stream()) == 0
    torch.cuda.synchronize()
    assert bool((got == 0).all()) and bool((dn == 0).all())
    c.weight[:] = 1.0
    c.dloss[:] = 1.0
    one = c.run()
    assert sat.rowop_distill(c.args(loss=got, dlogits=dn, ldd=100, weight=None, dloss=None), stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(one[0], got) and torch.equal(one[2], dn)


def test_offsets_past_32_bits():
    ld, rows, vocab = 1 << 28, 10, 40000
    big = torch.empty((rows - 1) * ld + vocab, device="cuda", dtype=torch.bfloat16)
    view = big.as_strided((rows, vocab), (ld, 1))
    c = Case(2, rows, vocab, 16, "bf16")
    loss, lse, d, _, _ = c.run()
    view.copy_(c.logits)
    assert sat.rowop_distill(c.args(logits=view, ldl=ld, loss=lse, dlogits=view, ldd=ld), stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(view, d) and torch.equal(loss, lse)


def test_on_another_stream():
    c = Case(2, 20, 50000, 16, "bf16")
    loss, lse, d, _, _ = c.run()
    side, got, e = torch.cuda.Stream(), torch.empty_like(loss), torch.empty_like(d)
    side.wait_stream(torch.cuda.current_stream())
    assert sat.rowop_distill(c.args(loss=got, dlogits=e, ldd=e.stride(0)), side.cuda_stream) == 0
    side.synchronize()
    assert torch.equal(loss, got) and torch.equal(d, e)


@pytest.mark.parametrize("tau,whole", [(1.0, False), (2.0, False), (1.5, True)])
def test_gradient_against_differences(tau, whole):
    # The loss's formula in 64 bits along a random direction of the logits; central differences of step 1e-4 are
    # within about 1e-8 of the derivative.
    c = Case(3, 4, 50, 7, "fp32", "fp32", tau, whole=whole)
    _, _, d, d2, _ = c.run()
    s, move = ref.f64(c.logits), np.random.default_rng(1).standard_normal((4, 50))
    other = (c.ids.cpu().numpy(), ref.f64(c.teacher), tau, ref.f64(c.weight), ref.f64(c.dloss),
             None if not whole else ref.f64(c.teacher_lse))
    up, down = (ref.distill(s + t * move, *other)[0] for t in (1e-4, -1e-4))
    slope = (ref.f64(c.dloss) * (up - down) / 2e-4).sum()
    for g in (d, d2):
        terms = ref.f64(g) * move
        assert abs(terms.sum() - slope) <= 2e-5 * np.abs(terms).sum()
