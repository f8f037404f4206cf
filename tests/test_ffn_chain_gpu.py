"""Feed-forward operators one after another without a synchronisation between
them, on data that change from step to step: kernels start while the one before
them ends, so each has to wait for what it reads, and nothing may be written
while it is still read. Every step's results are those of the same calls one at
a time, bit by bit."""
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import ffn_reference as ref
from tests.gpu_util import stream

pytestmark = pytest.mark.gpu

STEPS = 12


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


class Training:
    """Forward with the pre-activations kept, backward from these (or computing them again) and both passes' workspace shared
    by all steps."""

    def __init__(self, rows, width, hidden, by_output, recompute, pad):
        g = torch.Generator(device="cuda")
        g.manual_seed(rows)
        shape = (2 * hidden, width) if by_output else (width, 2 * hidden)

        def inputs():
            return [ref.rows(g, rows, width, "fp16", pad), ref.rows(g, *shape, "fp16", pad, scale=width**-0.5),
                    ref.rows(g, rows, hidden, "fp16", pad)]

        self.sets, self.now = [inputs() for _ in range(3)], inputs()
        x, w, dh = self.now
        self.outputs = [ref.rows(g, rows, hidden, "fp16", pad), ref.rows(g, rows, 2 * hidden, "fp16", pad),
                        ref.rows(g, rows, width, "fp16", pad), ref.rows(g, *shape, "fp32", pad)]
        h, pre, dx, dw = self.outputs
        f = dict(rows=rows, width=width, hidden=hidden, type="fp16", activation="gelu", w_by_output=int(by_output), x=x,
                 ldx=x.stride(0), w=w, ldw=w.stride(0))
        self.forward = sat.FfnArgs(h=h, ldh=h.stride(0), preact=pre, ldp=pre.stride(0), **f)
        self.again = sat.FfnArgs(**f, **({} if recompute else dict(preact=pre, ldp=pre.stride(0))))
        self.grads = sat.FfnGrads(dh=dh, lddh=dh.stride(0), dx=dx, lddx=dx.stride(0), dw=dw, lddw=dw.stride(0), dw_type="fp32")
        size = sat.ffn_gated_workspace(self.forward), sat.ffn_gated_backward_workspace(self.again, self.grads)
        self.workspace = torch.empty(max(size), device="cuda", dtype=torch.uint8)
        self.forward.workspace = self.grads.workspace = self.workspace
        self.forward.workspace_bytes = self.grads.workspace_bytes = max(size)

    def step(self, i):
        for to, new in zip(self.now, self.sets[i % 3]):
            to.copy_(new)
        assert sat.ffn_gated(self.forward, stream()) == 0, sat.gemm_last_error()
        assert sat.ffn_gated_backward(self.again, self.grads, stream()) == 0, sat.gemm_last_error()
        return [t.clone() for t in self.outputs]

    def poison(self):
        for t in self.outputs:
            t.fill_(float("nan"))


class Serving:
    """Values from four bits and back to four bits, then products of these, gated and plain; rows off 16 bytes between them."""

    def __init__(self, rows, width, hidden, pad):
        g = torch.Generator(device="cuda")
        g.manual_seed(rows)

        def microscaled(n, m):
            return (torch.zeros(n, -(-m // 32) * 16, device="cuda", dtype=torch.uint8),
                    torch.zeros(sat.mxfp4_scale_bytes(n, m), device="cuda", dtype=torch.uint8))

        def quantising(values, to):
            n, m = values.shape
            return sat.Mxfp4Args(rows=n, width=m, type="bf16", values=values, ldv=values.stride(0), codes=to[0], ldc=to[0].stride(0),
                                 scales=to[1])

        def product(a, b, out, m, n, k, up=None):
            f = dict(up_codes=up[0], ldu=up[0].stride(0), up_scales=up[1], activation="silu") if up else {}
            return sat.Mxfp4GemmArgs(rows=m, cols=n, width=k, out_type="bf16", alpha=1.0, a_codes=a[0], lda=a[0].stride(0), a_scales=a[1],
                                     b_codes=b[0], ldb=b[0].stride(0), b_scales=b[1], out=out, ldo=out.stride(0), **f)

        def stored(n, m, scale):
            to = microscaled(n, m)
            sat.check(sat.mxfp4_quantize(quantising(ref.rows(g, n, m, "bf16", scale=scale), to), stream()))
            return to

        self.sets, self.now = [stored(rows, width, 1.0) for _ in range(3)], microscaled(rows, width)
        gate, up, down = stored(hidden, width, width**-0.5), stored(hidden, width, width**-0.5), stored(width, hidden, hidden**-0.5)
        x, h, y = (ref.rows(g, rows, n, "bf16", pad, pad) for n in (width, hidden, width))
        x4, h4 = microscaled(rows, width), microscaled(rows, hidden)
        self.outputs = [x, h, y, *x4, *h4]
        self.calls = [(sat.mxfp4_dequantize, quantising(x, self.now)), (sat.mxfp4_quantize, quantising(x, x4)),
                      (sat.mxfp4_gemm, product(x4, gate, h, rows, hidden, width, up)), (sat.mxfp4_quantize, quantising(h, h4)),
                      (sat.mxfp4_gemm, product(h4, down, y, rows, width, hidden))]

    def step(self, i):
        for to, new in zip(self.now, self.sets[i % 3]):
            to.copy_(new)
        for call, args in self.calls:
            assert call(args, stream()) == 0, sat.gemm_last_error()
        return [t.clone() for t in self.outputs]

    def poison(self):
        for t in self.outputs:
            t.fill_(float("nan") if t.is_floating_point() else 0xA5)


def check(run):
    want = []
    for i in range(3):
        run.poison()
        want.append(run.step(i))
        torch.cuda.synchronize()

    def same(got):
        torch.cuda.synchronize()
        for i, outs in enumerate(got):
            for n, (a, b) in enumerate(zip(outs, want[i % 3])):
                assert torch.equal(a, b), f"output {n} of step {i}"

    run.poison()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        same([run.step(i) for i in range(STEPS)])
    run.poison()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [run.step(i) for i in range(STEPS)]
    for _ in range(3):
        graph.replay()
    same(got)


@pytest.mark.parametrize("pad", [3, 0])
@pytest.mark.parametrize("recompute", [False, True])
@pytest.mark.parametrize("by_output", [True, False])
@pytest.mark.parametrize("rows,width,hidden", [(515, 1001, 2003), (7, 129, 301), (66, 1030, 33), (1, 40, 520), (2050, 200, 130)])
def test_training_steps(rows, width, hidden, by_output, recompute, pad):
    check(Training(rows, width, hidden, by_output, recompute, pad))


@pytest.mark.parametrize("pad", [3, 0])
@pytest.mark.parametrize("rows,width,hidden", [(515, 1001, 2003), (7, 129, 301), (1, 4096, 1000), (2050, 200, 130)])
def test_serving_steps(rows, width, hidden, pad):
    check(Serving(rows, width, hidden, pad))
