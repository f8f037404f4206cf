"""The feed-forward operators' bounded waits, in a library of their own built so
that a wait gives up at its first look, while what it is for is mostly still on
its way. The results are then NaN and never half made: every output element is
NaN or as it should be, nothing is left unwritten, nothing is written beside it,
and the calls come back and leave the device usable."""
import ctypes
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import ffn_reference as ref
from tests.gpu_util import stream
from tests.test_mxfp4_gpu import Product

sat_build = sys.modules["shape_adaptive_tile_gb300.build"]

pytestmark = pytest.mark.gpu

REST = r'''
namespace sat {
void set_last_error(const char*) {}
int fail_with(int code, const char*, ...) { return code; }
}  // namespace sat
'''


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    """The calls of a build that waits for nothing."""
    torch.cuda.set_device(0)
    sat.build()
    at = tmp_path_factory.mktemp("impatient")
    (at / "rest.cu").write_text(REST)
    sources = [os.path.join(sat_build.CSRC, f) for f in
               ("ffn.cu", "ffn_tiles_half.cu", "ffn_tiles_grad.cu", "ffn_tiles_mx.cu", "tensor_map.cpp")] + [str(at / "rest.cu")]

    def compiled(src):
        obj = str(at / (os.path.basename(src) + ".o"))
        # Its own statics, where both libraries are loaded.
        subprocess.run([sat_build._nvcc(), *sat_build.FLAGS, "-Xcompiler", "-fno-gnu-unique", "-DSAT_FFN_WAIT_NS=0", "-c", src,
                        "-o", obj], check=True)
        return obj

    with ThreadPoolExecutor() as pool:
        objects = list(pool.map(compiled, sources))
    subprocess.run([sat_build._nvcc(), *sat_build.ARCH, "-shared", "-o", str(at / "ffn.so"), *objects], check=True)
    lib = ctypes.CDLL(str(at / "ffn.so"))
    lib.ffn_gated.argtypes = lib.mxfp4_gemm.argtypes = [ctypes.c_void_p] * 2
    lib.ffn_gated_backward.argtypes = [ctypes.c_void_p] * 3
    return lib


def given_up(got, good):
    """How many elements are NaN; the others have to be what the library's call gives, bit by bit."""
    lost = 0
    for a, b in zip(got, good):
        nan = a.isnan()
        assert torch.equal(torch.where(nan, torch.zeros_like(a), a), torch.where(nan, torch.zeros_like(b), b))
        lost += int(nan.sum())
    return lost


def out(g, rows, width, kind, pad):
    """Zeros where a call has to write, NaN around them."""
    return ref.rows(g, rows, width, kind, pad, pad).zero_()


def inside_only(*ts):
    torch.cuda.synchronize()
    assert all(bool(torch.isnan(ref.surroundings(t)).all()) for t in ts), "wrote outside"


@pytest.mark.parametrize("by_output", [True, False])
@pytest.mark.parametrize("rows,width,hidden,pad", [(1, 4096, 640, 0), (48, 2048, 520, 1), (200, 1024, 320, 0), (700, 512, 1600, 3),
                                                   (2700, 328, 2056, 0)])
def test_gated_product_and_its_gradients(impatient, rows, width, hidden, pad, by_output):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = ref.rows(g, rows, width, "bf16")
    w = ref.rows(g, *((2 * hidden, width) if by_output else (width, 2 * hidden)), "bf16", scale=width**-0.5)
    dh = ref.rows(g, rows, hidden, "bf16")

    def run(forward, backward):
        h, pre = out(g, rows, hidden, "bf16", pad), out(g, rows, 2 * hidden, "bf16", pad)
        dx, dw = out(g, rows, width, "bf16", pad), out(g, *w.shape, "fp32", pad)
        args = sat.FfnArgs(rows=rows, width=width, hidden=hidden, type="bf16", activation="silu", w_by_output=int(by_output), x=x,
                           ldx=width, w=w, ldw=w.stride(0), h=h, ldh=h.stride(0), preact=pre, ldp=pre.stride(0))
        size = sat.ffn_gated_workspace(args)
        args.workspace, args.workspace_bytes = torch.zeros(max(size, 16), device="cuda", dtype=torch.uint8), size
        assert forward(args.address, stream()) == 0
        again = sat.FfnArgs(rows=rows, width=width, hidden=hidden, type="bf16", activation="silu", w_by_output=int(by_output), x=x,
                            ldx=width, w=w, ldw=w.stride(0))
        grads = sat.FfnGrads(dh=dh, lddh=hidden, dx=dx, lddx=dx.stride(0), dw=dw, lddw=dw.stride(0), dw_type="fp32")
        size = sat.ffn_gated_backward_workspace(again, grads)
        grads.workspace, grads.workspace_bytes = torch.zeros(size, device="cuda", dtype=torch.uint8), size
        assert backward(again.address, grads.address, stream()) == 0
        inside_only(h, pre, dx, dw)
        return h, pre, dx, dw

    good = run(sat.lib().ffn_gated, sat.lib().ffn_gated_backward)
    assert given_up(good, good) == 0
    assert given_up(run(impatient.ffn_gated, impatient.ffn_gated_backward), good) > 0
    assert given_up(run(sat.lib().ffn_gated, sat.lib().ffn_gated_backward), good) == 0


@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("rows,cols,width,kind", [(1, 1024, 8192, "bf16"), (40, 300, 4096, "fp32"), (200, 600, 1000, "fp16"),
                                                  (2600, 2600, 512, "bf16"), (2600, 2600, 512, "fp32")])
def test_products_of_microscaled_matrices(impatient, rows, cols, width, kind, activation):
    p = Product(2, rows, cols, width, kind, activation, pad=1)

    def run(call):
        o = out(p.g, rows, cols, kind, 1)
        args = p.args(o)
        assert call(args.address, stream()) == 0
        inside_only(o)
        return (o,)

    good = run(sat.lib().mxfp4_gemm)
    assert given_up(run(impatient.mxfp4_gemm), good) > 0
    assert given_up(run(sat.lib().mxfp4_gemm), good) == 0
