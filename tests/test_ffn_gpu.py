"""The gated product of the feed-forward block and its gradients against their
definitions in 64 bits."""
import numpy as np
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import ffn_reference as ref
from tests.gpu_util import stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


def scratch(size):
    return torch.empty(max(size, 16), device="cuda", dtype=torch.uint8) if size else None


class Case:
    def __init__(self, seed, rows, width, hidden, kind="bf16", activation="silu", by_output=True, pad=0, offset=0, out_pad=0,
                 out_offset=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.kind, self.activation, self.by_output = g, kind, activation, by_output
        self.rows, self.width, self.hidden, self.out_pad, self.out_offset = rows, width, hidden, out_pad, out_offset
        self.x = ref.rows(g, rows, width, kind, pad, offset)
        shape = (2 * hidden, width) if by_output else (width, 2 * hidden)
        self.w = ref.rows(g, *shape, kind, pad, offset, 1.5 * max(width, 1)**-0.5)
        self.dh = ref.rows(g, rows, hidden, kind, pad, offset)
        self.pad, self.offset = pad, offset

    def out(self, n, width, kind):
        return ref.rows(self.g, n, width, kind, self.out_pad, self.out_offset).fill_(float("nan"))

    def args(self, **more):
        f = dict(rows=self.rows, width=self.width, hidden=self.hidden, type=self.kind, activation=self.activation,
                 w_by_output=int(self.by_output), x=self.x, ldx=self.x.stride(0), w=self.w, ldw=self.w.stride(0))
        return sat.FfnArgs(**{**f, **more})

    def forward(self, keep=False, to=None, **more):
        h = self.out(self.rows, self.hidden, self.kind)
        pre = self.out(self.rows, 2 * self.hidden, self.kind) if keep else None
        a = self.args(h=h, ldh=h.stride(0), preact=pre, ldp=pre.stride(0) if keep else 0, **more)
        size = sat.ffn_gated_workspace(a)
        a.workspace, a.workspace_bytes = scratch(size), size
        assert sat.ffn_gated(a, stream() if to is None else to) == 0, sat.gemm_last_error()
        torch.cuda.synchronize()
        for t in (h, pre):
            if t is not None:
                assert bool(torch.isnan(ref.surroundings(t)).all()), "wrote outside"
        return h, pre

    def check_forward(self, keep=False):
        p = ref.Gated(self.x, self.w, self.by_output, self.hidden)
        h, pre = self.forward(keep)
        ref.assert_within(h, *p.h(self.kind, self.activation), "h")
        if keep:
            z, off = torch.cat([p.g, p.u], 1), torch.cat([p.dg, p.du], 1)
            ref.assert_within(pre, z, off + ref.half_step(z.abs() + off, self.kind), "preact")
        return h

    def backward(self, preact=None, dw_kind=None, into=None, dx=True, dw=True, to=None):
        dw_kind = dw_kind or self.kind
        gx = self.out(self.rows, self.width, self.kind) if dx else None
        gw = (self.out(*self.w.shape, dw_kind) if into is None else into) if dw else None
        a = self.args(preact=preact, ldp=preact.stride(0) if preact is not None else 0)
        g = sat.FfnGrads(dh=self.dh, lddh=self.dh.stride(0), dx=gx, lddx=gx.stride(0) if dx else 0, dw=gw,
                         lddw=gw.stride(0) if dw else 0, dw_type=dw_kind, accumulate=int(into is not None))
        size = sat.ffn_gated_backward_workspace(a, g)
        g.workspace, g.workspace_bytes = scratch(size), size
        assert sat.ffn_gated_backward(a, g, stream() if to is None else to) == 0, sat.gemm_last_error()
        torch.cuda.synchronize()
        for t in (gx, gw if into is None else None):
            if t is not None:
                assert bool(torch.isnan(ref.surroundings(t)).all()), "wrote outside"
        return gx, gw

    def check_backward(self, recompute, dw_kind=None, accumulate=False):
        dw_kind = dw_kind or self.kind
        preact = None
        if not recompute:
            p = ref.Gated(self.x, self.w, self.by_output, self.hidden)
            preact = ref.rows(self.g, self.rows, 2 * self.hidden, self.kind, self.pad, self.offset)
            preact.copy_(torch.cat([p.g, p.u], 1))
        into, before = None, 0.0
        if accumulate:
            into = ref.rows(self.g, *self.w.shape, dw_kind, self.out_pad, self.out_offset)
            before = into.double().clone()
        gx, gw = self.backward(preact, dw_kind, into)
        dx, off_dx, dw, off_dw = ref.gradients(self.x, self.w, self.by_output, self.hidden, self.kind, self.activation,
                                               self.dh, preact)
        ref.assert_within(gx, dx, off_dx + ref.half_step(dx.abs() + off_dx, self.kind), "dx")
        dw = dw + before
        off_dw = off_dw + ref.half_step(dw.abs() + off_dw, dw_kind)
        ref.assert_within(gw, dw, off_dw, "dw")


SIZES = [(1, 64, 128), (1, 8, 8), (1, 1, 1), (2, 1000, 333), (16, 256, 640), (17, 72, 136), (33, 512, 1024), (64, 2048, 256),
         (65, 136, 200), (128, 64, 64), (129, 264, 130), (300, 1032, 72), (257, 513, 385), (640, 320, 1920), (1000, 128, 2504),
         (70, 4096, 64)]


@pytest.mark.parametrize("by_output", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,width,hidden", SIZES)
def test_forward_sizes(rows, width, hidden, kind, by_output):
    Case(rows + hidden, rows, width, hidden, kind, by_output=by_output).check_forward()
    Case(rows + hidden, rows, width, hidden, kind, "gelu_tanh", by_output).check_forward(keep=True)


@pytest.mark.parametrize("activation", ["none", "silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("rows", [5, 200])
def test_activations(rows, activation):
    c = Case(3, rows, 256, 264, "bf16", activation)
    c.check_forward(keep=True)
    c.check_backward(True)
    c.check_backward(False)


@pytest.mark.parametrize("recompute", [True, False])
@pytest.mark.parametrize("by_output", [True, False])
@pytest.mark.parametrize("rows,width,hidden", SIZES)
def test_backward_sizes(rows, width, hidden, by_output, recompute):
    Case(rows + hidden, rows, width, hidden, "bf16", "silu", by_output).check_backward(recompute)
    Case(rows + hidden, rows, width, hidden, "fp16", "gelu", by_output).check_backward(recompute, "fp32")


@pytest.mark.parametrize("by_output", [True, False])
def test_weight_gradients_accumulate(by_output):
    Case(1, 200, 136, 72, "bf16", "silu", by_output).check_backward(True, "fp32", accumulate=True)
    Case(1, 200, 136, 72, "fp16", "silu", by_output, out_pad=3, out_offset=1).check_backward(False, "fp32", accumulate=True)


@pytest.mark.parametrize("i", range(24))
def test_strides_and_alignment(i):
    rng = np.random.default_rng(100 + i)
    rows, width, hidden = (int(2**rng.uniform(0, t)) for t in (9, 9, 9))
    c = Case(i, rows, width, hidden, ("bf16", "fp16")[i % 2], ("silu", "gelu", "relu")[i % 3], bool(rng.integers(2)),
             int(rng.choice([0, 1, 3, 8])), int(rng.choice([0, 1, 3, 8])), int(rng.choice([0, 1, 3, 8])),
             int(rng.choice([0, 1, 3, 8])))
    c.check_forward(keep=bool(rng.integers(2)))
    c.check_backward(bool(rng.integers(2)))


@pytest.mark.parametrize("out_pad,out_offset", [(0, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("by_output", [True, False])
@pytest.mark.parametrize("rows,width,hidden", [(66, 1030, 33), (70, 2056, 200), (129, 4096, 104), (96, 16400, 72), (200, 9000, 1)])
def test_long_sums_of_few_outputs(rows, width, hidden, by_output, out_pad, out_offset):
    """Tiles that several CTAs share: whole and ragged chunks of columns, rows on and off 16 bytes."""
    c = Case(rows + hidden, rows, width, hidden, "bf16", "silu", by_output, out_pad=out_pad, out_offset=out_offset)
    c.check_forward(keep=True)
    c.check_forward()
    c.check_backward(True)
    c.check_backward(False)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("by_output", [True, False])
@pytest.mark.parametrize("rows,width,hidden,out_pad", [(4100, 130, 50, 0), (9000, 72, 36, 1), (2050, 200, 130, 4)])
def test_weight_gradients_of_many_rows(rows, width, hidden, out_pad, by_output, accumulate):
    c = Case(rows + hidden, rows, width, hidden, "fp16", "gelu_tanh", by_output, out_pad=out_pad)
    c.check_backward(True, "fp32", accumulate)
    if not accumulate:
        c.check_backward(False, "fp16")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_many_tiles(kind):
    # More tiles than SMs: several rounds of the persistent kernels, in both directions along k.
    c = Case(1, 2700, 328, 2056, kind, "silu")
    c.check_forward(keep=True)
    c.check_backward(True)
    c = Case(2, 2700, 1032, 2056, kind, "gelu_tanh", False)
    c.check_forward()
    c.check_backward(False)


@pytest.mark.parametrize("hidden", [70, 193, 333])
def test_rows_on_16_bytes_whose_last_piece_is_not_whole(hidden):
    for rows in (20, 300):
        for by_output in (True, False):
            c = Case(3, rows, 100 + hidden, hidden, "bf16", by_output=by_output, out_pad=-hidden % 8)
            c.check_forward(keep=True)
            c.out_pad = -c.width % 8
            c.check_backward(True)
            c.check_backward(False, "fp32")


def test_empty_sizes():
    for by_output in (True, False):
        for size in ((0, 64, 64), (5, 0, 24), (5, 24, 0)):
            c = Case(1, *size, by_output=by_output)
            h, pre = c.forward(keep=True)
            assert not h.any() and not pre.any()  # nothing there, or products of nothing
            gx, gw = c.backward(pre)
            assert not gx.any() and not gw.any()
    c = Case(1, 0, 24, 16)
    into = torch.ones(32, 24, device="cuda")
    c.backward(None, "fp32", into)
    assert bool((into == 1).all())


def test_parts_of_the_gradient():
    c = Case(4, 150, 264, 200)
    gx, gw = c.backward()
    assert torch.equal(c.backward(dw=False)[0], gx)
    assert torch.equal(c.backward(dx=False)[1], gw)
    assert c.backward(dx=False, dw=False) == (None, None)


def test_gradients_against_differences():
    # The loss is sum h dh; along a direction its slope is that of (h(+) - h(-)) / 2 s, in 64 bits from the definition: what is
    # checked is that dx and dw are gradients of the forward formula. The difference is exact to s^2 times third derivatives
    # (well below 1e-5 of the sum here), the gradients to their tolerances.
    for activation in ("silu", "gelu", "gelu_tanh"):
        c = Case(6, 40, 72, 48, "fp16", activation)
        gx, gw = c.backward(dw_kind="fp32")
        vx = torch.randn(c.x.shape, device="cuda", generator=c.g, dtype=torch.float64)
        vw = torch.randn(c.w.shape, device="cuda", generator=c.g, dtype=torch.float64) * 0.1
        dx, off_dx, dw, off_dw = ref.gradients(c.x, c.w, True, 48, "fp16", activation, c.dh)
        off_dx, off_dw = off_dx + ref.half_step(dx.abs() + off_dx, "fp16"), off_dw + ref.half_step(dw.abs() + off_dw, "fp32")

        def loss(step_x, step_w):
            p = ref.Gated(c.x.double() + step_x * vx, c.w.double() + step_w * vw, True, 48)
            return float((ref.act(p.g, activation)[0] * p.u * c.dh.double()).sum())

        s = 1e-4
        for got, v, off, slope in ((gx, vx, off_dx, (loss(s, 0) - loss(-s, 0)) / (2 * s)),
                                   (gw, vw, off_dw, (loss(0, s) - loss(0, -s)) / (2 * s))):
            assert abs(float((got.double() * v).sum()) - slope) <= float((off * v.abs()).sum()) + 1e-4


def test_not_a_number_stays_in_its_row():
    for rows in (3, 200):
        c = Case(9, rows, 128, 136, "bf16")
        clean = c.forward()[0].clone()
        c.x[1, 5] = float("nan")
        c.x[2, 7] = float("inf")
        h = c.forward()[0]
        assert bool(torch.isnan(h[1]).all()) and not bool(torch.isfinite(h[2]).any())
        keep = [r for r in range(rows) if r not in (1, 2)]
        assert torch.equal(h[keep], clean[keep])


def test_results_repeat_and_follow_the_stream():
    for rows, width, hidden in ((1, 2048, 1024), (48, 1000, 512), (700, 512, 1600)):
        c = Case(8, rows, width, hidden)
        h = c.forward()[0].clone()
        gx, gw = c.backward()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            assert torch.equal(c.forward(to=side.cuda_stream)[0], h)
            again = c.backward(to=side.cuda_stream)
            assert torch.equal(again[0], gx) and torch.equal(again[1], gw)


def test_captured_into_a_graph():
    c = Case(8, 300, 520, 640)
    h, pre = c.out(300, 640, "bf16"), c.out(300, 1280, "bf16")
    gx, gw = c.out(300, 520, "bf16"), c.out(1280, 520, "fp32")
    a = c.args(h=h, ldh=h.stride(0), preact=pre, ldp=pre.stride(0))
    g = sat.FfnGrads(dh=c.dh, lddh=c.dh.stride(0), dx=gx, lddx=gx.stride(0), dw=gw, lddw=gw.stride(0), dw_type="fp32")
    size = sat.ffn_gated_backward_workspace(a, g)
    g.workspace, g.workspace_bytes = scratch(size), size
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert sat.ffn_gated(a, stream()) == 0 and sat.ffn_gated_backward(a, g, stream()) == 0, sat.gemm_last_error()
    for seed in (1, 2):
        new = Case(seed, 300, 520, 640)
        c.x.copy_(new.x), c.w.copy_(new.w), c.dh.copy_(new.dh)
        graph.replay()
        torch.cuda.synchronize()
        want, want_pre = c.forward(keep=True)
        assert torch.equal(h, want) and torch.equal(pre, want_pre)
        assert all(torch.equal(x, y) for x, y in zip((gx, gw), c.backward(want_pre, "fp32")))


def test_offsets_past_32_bits():
    ld = (1 << 30) + 8  # rows 2 GB apart
    c = Case(5, 5, 72, 40)
    want = c.forward()[0]
    big = torch.empty(4 * ld + 72, device="cuda", dtype=torch.bfloat16)
    x = big.as_strided((5, 72), (ld, 1))
    x.copy_(c.x)
    c.x = x
    assert torch.equal(c.forward()[0], want)
    out = torch.empty(4 * ld + 40, device="cuda", dtype=torch.bfloat16).as_strided((5, 40), (ld, 1))
    a = c.args(h=out, ldh=ld)
    assert sat.ffn_gated(a, stream()) == 0, sat.gemm_last_error()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_training_step_of_the_block():
    # Gated product, down projection, its gradients and the gated product's, with the library's own products between; each
    # step against the definition on what the step before it gave.
    rows, width, hidden = 384, 256, 640
    c = Case(3, rows, width, hidden, "bf16", "silu")
    down = ref.rows(c.g, hidden, width, "bf16", scale=hidden**-0.5)
    dy = ref.rows(c.g, rows, width, "bf16")
    h, pre = c.forward(keep=True)
    ref.assert_within(h, *ref.Gated(c.x, c.w, True, hidden).h("bf16", "silu"), "h")
    y, dh, ddown = (torch.empty(*s, device="cuda", dtype=torch.bfloat16) for s in ((rows, width), (rows, hidden), (hidden, width)))
    products = ((h, down, y, rows, width, hidden, False, False), (dy, down, dh, rows, hidden, width, False, True),
                (h, dy, ddown, hidden, width, rows, True, False))
    for a, b, to, m, n, k, ta, tb in products:
        with sat.Plan(m, n, k, "bf16", trans_a=ta, trans_b=tb, c_type="bf16") as plan:
            plan.run(a, b, to, 1.0, 0.0, stream())
            torch.cuda.synchronize()
        u, v = (a.double().t() if ta else a.double()), (b.double().t() if tb else b.double())
        want, off = u @ v, ref.sum_error(k, u.abs() @ v.abs())
        ref.assert_within(to, want, off + ref.half_step(want.abs() + off, "bf16"), "product")
    c.dh = dh
    gx, gw = c.backward(pre, "fp32")
    dx, off_dx, dw, off_dw = ref.gradients(c.x, c.w, True, hidden, "bf16", "silu", dh, pre)
    ref.assert_within(gx, dx, off_dx + ref.half_step(dx.abs() + off_dx, "bf16"), "dx")
    ref.assert_within(gw, dw, off_dw + ref.half_step(dw.abs() + off_dw, "fp32"), "dw")


def test_two_streams_at_once():
    cases = [Case(s, 515, 264, 1001, "fp16", "gelu", pad=3) for s in (1, 2)]
    want = [(c.forward()[0].clone(), *(t.clone() for t in c.backward())) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    runs = []
    for c in cases:  # buffers of each call's own
        h, gx, gw = c.out(515, 1001, "fp16"), c.out(515, 264, "fp16"), c.out(2002, 264, "fp16")
        a = c.args(h=h, ldh=h.stride(0))
        size = sat.ffn_gated_workspace(a)
        a.workspace, a.workspace_bytes = scratch(size), size
        b = c.args()
        g = sat.FfnGrads(dh=c.dh, lddh=c.dh.stride(0), dx=gx, lddx=gx.stride(0), dw=gw, lddw=gw.stride(0), dw_type="fp16")
        size = sat.ffn_gated_backward_workspace(b, g)
        g.workspace, g.workspace_bytes = scratch(size), size
        runs.append((a, b, g, (h, gx, gw)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (a, b, g, _) in zip(streams, runs):
            assert sat.ffn_gated(a, s.cuda_stream) == 0 and sat.ffn_gated_backward(b, g, s.cuda_stream) == 0
    torch.cuda.synchronize()
    for w, r in zip(want, runs):
        assert all(torch.equal(x, y) for x, y in zip(w, r[3]))


def test_the_first_call_of_a_process_may_be_a_captured_one():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(sat.__file__)))
    code = """
import torch, shape_adaptive_tile_gb300 as sat
x, w = torch.randn(300, 256, device="cuda").bfloat16(), torch.randn(1024, 256, device="cuda").bfloat16() / 16
h = torch.zeros(300, 512, device="cuda", dtype=torch.bfloat16)
a = sat.FfnArgs(rows=300, width=256, hidden=512, type="bf16", activation="none", w_by_output=1, x=x, ldx=256, w=w, ldw=256, h=h, ldh=512)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    sat.check(sat.ffn_gated(a, torch.cuda.current_stream().cuda_stream))
g.replay()
torch.cuda.synchronize()
z = x.double() @ w.double().t()
assert float((h.double() - z[:, :512] * z[:, 512:]).abs().max()) < 0.1
"""
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)


def test_the_first_call_of_a_process_may_be_a_captured_one_of_shared_tiles():
    """How many clusters the device holds is asked for by the first call, here while a graph is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(sat.__file__)))
    code = """
import torch, shape_adaptive_tile_gb300 as sat
x, w = torch.randn(96, 4096, device="cuda").bfloat16(), torch.randn(512, 4096, device="cuda").bfloat16() / 64
h, one = (torch.zeros(n, 256, device="cuda", dtype=torch.bfloat16) for n in (96, 1))
f = dict(width=4096, hidden=256, type="bf16", activation="none", w_by_output=1, x=x, ldx=4096, w=w, ldw=4096, ldh=256)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for n, out in ((96, h), (1, one)):
        sat.check(sat.ffn_gated(sat.FfnArgs(rows=n, h=out, **f), torch.cuda.current_stream().cuda_stream))
g.replay()
torch.cuda.synchronize()
z = x.double() @ w.double().t()
want = z[:, :256] * z[:, 256:]
assert float((h.double() - want).abs().max()) < 0.1 and float((one.double() - want[:1]).abs().max()) < 0.1
"""
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)
