"""Verification of drafted tokens against the rule in 64 bits.

Tokens have to be equal wherever the deciding numbers are apart by more than
1e-4 of their size (probabilities in fp32 are good to about 1e-5); such near
ties are rare, and the tests count them. Log-probabilities: 8e-6 + 3e-7 of the
logits' range.
"""
import numpy as np
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import lm_reference as ref
from tests.gpu_util import stream

pytestmark = pytest.mark.gpu

NEAR = 1e-4


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


class Case:
    def __init__(self, seed, batch, drafts, vocab, dtype="fp32", tau=1.0, draft_tau=None, point=False, ragged=False, pad=0,
                 offset=0, spread=2.5):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.batch, self.drafts, self.vocab, self.dtype, self.tau = batch, drafts, vocab, dtype, tau
        self.draft_tau = draft_tau or tau or 1.0

        def rows(v, kind):
            whole = torch.empty(offset + v.shape[0] * (vocab + pad) + 8, device="cuda", dtype=ref.TYPES[kind])
            view = whole[offset:offset + v.shape[0] * (vocab + pad)].view(v.shape[0], vocab + pad)[:, :vocab]
            return view.copy_(v)

        def normal(n):
            return torch.randn(n, vocab, device="cuda", generator=g)

        t = normal(batch * (drafts + 1)) * spread
        near = t.view(batch, drafts + 1, vocab)[:, :drafts].reshape(-1, vocab) + 0.7 * normal(batch * drafts)
        self.target = rows(t, dtype)
        self.draft = None if point else rows(near, dtype)
        race = torch.empty_like(near).exponential_(generator=g)
        self.tokens = (near / self.draft_tau - race.log()).argmax(-1).int().view(batch, drafts).contiguous() if drafts else None
        self.lengths = torch.randint(0, drafts + 1, (batch,), device="cuda", generator=g).int() if ragged else None
        self.uniforms = torch.rand(batch, drafts, device="cuda", generator=g) if drafts else None
        self.noise = rows(torch.empty(batch, vocab, device="cuda").exponential_(generator=g).clamp_(min=1e-20), "fp32")

    def args(self, **more):
        size = sat.rowop_verify_workspace(self.batch, self.drafts, self.vocab)
        f = dict(batch=self.batch, drafts=self.drafts, vocab=self.vocab, logits_type=self.dtype, temperature=self.tau,
                 draft_temperature=self.draft_tau, target=self.target, ldt=self.target.stride(0), draft=self.draft,
                 ldq=self.draft.stride(0) if self.draft is not None else 0, tokens=self.tokens, lengths=self.lengths,
                 uniforms=self.uniforms, noise=self.noise, ldn=self.noise.stride(0),
                 workspace=torch.empty(max(size, 1), device="cuda", dtype=torch.uint8), workspace_bytes=size)
        return sat.VerifyArgs(**{**f, **more})

    def run(self, **more):
        accepted = torch.full((self.batch,), -9, device="cuda", dtype=torch.int32)
        out = torch.full((self.batch, self.drafts + 1), -9, device="cuda", dtype=torch.int32)
        lp = torch.full((self.batch, self.drafts + 1), float("nan"), device="cuda")
        assert sat.rowop_verify(self.args(accepted=accepted, out=out, logprobs=lp, **more), stream()) == 0, sat.gemm_last_error()
        torch.cuda.synchronize()
        return accepted.cpu().numpy(), out.cpu().numpy(), ref.f64(lp)

    def check(self):
        got = self.run()
        tokens = np.zeros((self.batch, 0), int) if self.tokens is None else self.tokens.cpu().numpy()
        lengths = np.full(self.batch, self.drafts) if self.lengths is None else self.lengths.cpu().numpy()
        uniforms = None if self.uniforms is None else ref.f64(self.uniforms)
        accepted, out, lp, margin = ref.verify(
            ref.f64(self.target), None if self.draft is None else ref.f64(self.draft), tokens, lengths, uniforms,
            ref.f64(self.noise), self.tau, self.draft_tau)
        sure = margin > NEAR
        assert sure.sum() >= 0.9 * self.batch - 1
        assert np.array_equal(got[0][sure], accepted[sure])
        assert np.array_equal(got[1][sure], out[sure])
        t = ref.f64(self.target)
        span = np.ptp(np.where(np.isfinite(t), t, 0.0)) / (self.tau or 1.0)
        ref.assert_within(got[2][sure], lp[sure], 8e-6 + 3e-7 * span, "logprobs")
        return accepted


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("batch,drafts,vocab", [(1, 4, 32768), (1, 0, 1000), (3, 1, 7), (2, 3, 1), (5, 8, 999), (17, 5, 4097),
                                                (2, 64, 300), (9, 2, 65537), (1, 7, 262147), (200, 3, 130)])
def test_sizes_and_types(batch, drafts, vocab, dtype):
    for tau, point in ((1.0, False), (0.8, True), (0.0, False)):
        Case(vocab + batch, batch, drafts, vocab, dtype, tau, point=point).check()


@pytest.mark.parametrize("i", range(40))
def test_random_strides_lengths_and_temperatures(i):
    rng = np.random.default_rng(70 + i)
    vocab, drafts = int(2 ** rng.uniform(1, 16)), int(rng.integers(0, 9))
    Case(i, int(rng.integers(1, 40)), drafts, vocab, ("fp32", "bf16", "fp16")[i % 3], float(rng.choice([1.0, 0.5, 1.7, 0.0])),
         float(rng.choice([1.0, 0.7])), bool(rng.random() < 0.3), bool(rng.integers(2)), int(rng.choice([0, 1, 3, 8])),
         int(rng.choice([0, 1, 3, 8]))).check()


def test_a_large_batch():
    assert len(set(Case(3, 1500, 4, 600, "bf16", 1.0, ragged=True).check())) == 5  # every number of accepted tokens occurs


def test_equal_distributions_accept_everything():
    c = Case(2, 30, 6, 2000)
    c.draft.copy_(c.target.view(30, 7, 2000)[:, :6].reshape(180, 2000))
    c.uniforms.clamp_(max=0.9999)
    assert (c.run()[0] == 6).all()
    c.uniforms[:, 2] = 1.0  # u q < p fails only by a u outside its range: then p - q is nowhere positive, and p is drawn from
    accepted, out, _ = c.run()
    assert (accepted == 2).all() and (out[:, 2] >= 0).all()
    p = np.exp(ref.log_softmax(ref.f64(c.target).reshape(30, 7, 2000)[:, 2]))
    assert np.array_equal(out[:, 2], (p / ref.f64(c.noise)).argmax(1))


def test_disjoint_distributions_refuse_everything():
    c = Case(2, 30, 3, 2000, "bf16")
    c.target[:, :1000] = float("-inf")
    c.draft[:, 1000:] = float("-inf")
    c.tokens.random_(0, 1000)
    assert (c.check() == 0).all()


@pytest.mark.parametrize("tau", [1.0, 0.0])
@pytest.mark.parametrize("vocab", [600, 40000])
def test_masks_and_rows_without_a_distribution(vocab, tau):
    c = Case(5, 12, 3, vocab, "fp32", tau)
    t = c.target.view(12, 4, vocab)
    t[0, :, vocab // 2:] = float("-inf")
    t[1, 0] = float("-inf")               # nothing allowed at the first token
    t[2, 1, 5] = float("nan")
    t[3, 3, 17] = float("inf")
    t[4, :] = torch.finfo(torch.float32).min
    t[5, :, 1:] = torch.finfo(torch.float32).min
    c.tokens[6, 0] = -1                   # outside the vocabulary
    c.tokens[7, 1] = vocab
    c.tokens[8, 2] = 2 ** 31 - 1
    c.lengths = torch.tensor([3, 3, 3, 3, 0, 2, 3, 3, 3, -4, 99, 1], device="cuda", dtype=torch.int32)
    if tau:
        c.uniforms[2:4] = 0.0             # accept what has any probability
    else:
        best = t.argmax(-1)[:, :3].int()
        c.tokens[2:4] = best[2:4]
    accepted, out, lp = c.run()
    assert accepted[1] == 0 and out[1, 0] == -1 and lp[1, 0] == 0
    assert accepted[2] == 1 and out[2, 1] == -1 and lp[2, 1] == 0
    assert accepted[3] == 3 and out[3, 3] == -1
    assert accepted[4] == 0 and accepted[9] == 0
    if tau == 0:
        assert out[4, 0] == 0 and out[5, 0] == 0  # ties go to the lowest token
    assert (out[np.arange(12) != 1, 0] >= 0).all()
    keep = [0, 5, 6, 7, 8, 9, 10, 11]
    tokens, lengths = c.tokens.cpu().numpy(), c.lengths.cpu().numpy()
    rows = np.concatenate([np.arange(b * 4, b * 4 + 4) for b in keep])
    drows = np.concatenate([np.arange(b * 3, b * 3 + 3) for b in keep])
    want = ref.verify(ref.f64(c.target)[rows], ref.f64(c.draft)[drows], tokens[keep], lengths[keep], ref.f64(c.uniforms)[keep],
                      ref.f64(c.noise)[keep], tau, c.draft_tau)
    sure = want[3] > NEAR
    assert np.array_equal(accepted[keep][sure], want[0][sure]) and np.array_equal(out[keep][sure], want[1][sure])


def test_greedy_takes_the_lowest_of_equals():
    c = Case(1, 6, 2, 5000, "bf16", 0.0)
    c.target[:] = c.target.clamp(max=1.0)  # many at the largest value
    t = c.target.view(6, 3, 5000)
    first = (t == t.amax(-1, keepdim=True)).int().argmax(-1)
    c.tokens.copy_(first[:, :2])
    accepted, out, _ = c.run()
    assert (accepted == 2).all() and np.array_equal(out, first.cpu().numpy())
    c.tokens[:, 1] += 1  # another of the equals, or none: refused
    assert (c.run()[0] == 1).all()
    assert sat.rowop_verify(c.args(accepted=c.tokens, out=c.tokens, noise=None, uniforms=None, batch=0), stream()) == 0


def test_inputs_of_other_modes_are_not_read():
    # Greedy: no random numbers and no draft; no logprobs: none written.
    c = Case(1, 4, 3, 999, "fp16", 0.0)
    accepted, out, _ = c.run()
    got, out2 = torch.empty(4, device="cuda", dtype=torch.int32), torch.empty(4, 4, device="cuda", dtype=torch.int32)
    assert sat.rowop_verify(c.args(accepted=got, out=out2, noise=None, uniforms=None, draft=None, ldn=0, ldq=0), stream()) == 0
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), accepted) and np.array_equal(out2.cpu().numpy(), out)


def test_results_repeat_and_follow_the_stream():
    c = Case(8, 33, 4, 20001, "bf16", 0.9, ragged=True)
    one = c.run()
    for _ in range(5):
        assert all(np.array_equal(a, b) for a, b in zip(one, c.run()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    accepted, out = torch.empty(33, device="cuda", dtype=torch.int32), torch.empty(33, 5, device="cuda", dtype=torch.int32)
    args = c.args(accepted=accepted, out=out)
    assert sat.rowop_verify(args, side.cuda_stream) == 0
    side.synchronize()
    assert np.array_equal(accepted.cpu().numpy(), one[0]) and np.array_equal(out.cpu().numpy(), one[1])


def test_offsets_past_32_bits():
    ld, batch, drafts, vocab = 1 << 28, 3, 2, 3000
    big = torch.empty((batch * (drafts + 1) - 1) * ld + vocab, device="cuda", dtype=torch.bfloat16)
    view = big.as_strided((batch * (drafts + 1), vocab), (ld, 1))
    c = Case(8, batch, drafts, vocab, "bf16")
    one = c.run()
    view.copy_(c.target)
    assert all(np.array_equal(a, b) for a, b in zip(one, c.run(target=view, ldt=ld)))


def test_the_tokens_are_distributed_as_the_target():
    # One pair of distributions for many sequences: the first token said, drafted or drawn, follows the target, and
    # the second, where the first was accepted, its own row. Five standard deviations of each frequency.
    batch, drafts, vocab = 200000, 2, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    t = torch.randn(drafts + 1, vocab, device="cuda", generator=g) * 1.2
    q = torch.randn(drafts, vocab, device="cuda", generator=g) * 1.2
    c = Case(4, batch, drafts, vocab)
    c.target.copy_(t.repeat(batch, 1))
    c.draft.copy_(q.repeat(batch, 1))
    race = torch.empty(batch, drafts, vocab, device="cuda").exponential_(generator=g)
    c.tokens.copy_((q - race.log()).argmax(-1))
    accepted, out, _ = c.run()
    p = np.exp(ref.log_softmax(ref.f64(t)))
    for i in range(drafts + 1):
        said = out[accepted >= i, i]
        freq = np.bincount(said, minlength=vocab) / len(said)
        assert (np.abs(freq - p[i]) <= 5 * np.sqrt(p[i] * (1 - p[i]) / len(said))).all()
