"""The feed-forward operators' bounded waits where they run out just as what they
wait for comes: of one tile's warps some then give up and others have their
sums. Every output element is NaN or as it should be all the same. A library of
their own, built with a limit of some microseconds, and sums so long that a
tile takes about as long as that."""
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
from tests.test_ffn_waits_gpu import REST

sat_build = sys.modules["shape_adaptive_tile_gb300.build"]

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    torch.cuda.set_device(0)
    sat.build()
    at = tmp_path_factory.mktemp("hasty")
    (at / "rest.cu").write_text(REST)
    sources = [os.path.join(sat_build.CSRC, f) for f in
               ("ffn.cu", "ffn_tiles_half.cu", "ffn_tiles_grad.cu", "ffn_tiles_mx.cu", "tensor_map.cpp")] + [str(at / "rest.cu")]

    def compiled(src):
        obj = str(at / (os.path.basename(src) + ".o"))
        subprocess.run([sat_build._nvcc(), *sat_build.FLAGS, "-Xcompiler", "-fno-gnu-unique", "-DSAT_FFN_WAIT_NS=8000", "-c", src,
                        "-o", obj], check=True)
        return obj

    with ThreadPoolExecutor() as pool:
        objects = list(pool.map(compiled, sources))
    subprocess.run([sat_build._nvcc(), *sat_build.ARCH, "-shared", "-o", str(at / "ffn.so"), *objects], check=True)
    lib = ctypes.CDLL(str(at / "ffn.so"))
    lib.ffn_gated.argtypes = lib.mxfp4_gemm.argtypes = [ctypes.c_void_p] * 2
    lib.ffn_gated_backward.argtypes = [ctypes.c_void_p] * 3
    return lib


def near_the_limit(make, shortest, longest):
    """Runs calls of sums of various lengths, and many around the length at which waits begin to run out. `make(k)` gives a
    call and its outputs by the library."""

    def lost(k, times):
        run, good = make(k)
        most = 0
        for _ in range(times):
            for got, want in zip(run(), good):
                nan = got.isnan()
                off = ~nan & (got != want)
                assert not bool(off.any()), f"k {k}: {int(off.sum())} elements are neither NaN nor right"
                most = max(most, int(nan.sum()))
        return most

    assert lost(longest, 2) > 0
    low, high = shortest, longest
    while high - low > 64:
        k = (low + high) // 128 * 64
        low, high = (k, high) if lost(k, 2) == 0 else (low, k)
    for k in range(max(shortest, high - 8 * 64), high + 9 * 64, 64):
        lost(k, 8)


def bytes_of(g, n, m, low=0, high=256):
    return torch.randint(low, high, (n, m), device="cuda", generator=g, dtype=torch.uint8)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols", [(5000, 5000), (200, 300), (30, 1000)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_products_of_microscaled_matrices(hasty, rows, cols, kind, gated):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)

    def make(k):
        a, b, c = (bytes_of(g, n, k // 2) for n in (rows, cols, cols))
        scales = [bytes_of(g, sat.mxfp4_scale_bytes(n, k), 1, 110, 120) for n in (rows, cols, cols)]
        for s, n in zip(scales, (rows, cols, cols)):  # (0 past the last row and block)
            s = s.view(-1, -(-k // 128), 32, 4, 4)
            r = torch.arange(s.shape[0] * 128, device="cuda").view(-1, 4, 32).permute(0, 2, 1)[:, None, :, :, None] >= n
            blocks = torch.arange(s.shape[1] * 4, device="cuda").view(1, -1, 1, 1, 4) >= k // 32
            s.masked_fill_(r | blocks, 0)
        out = torch.empty(rows, cols, device="cuda", dtype=ref.TYPES[kind])
        f = dict(up_codes=c, ldu=k // 2, up_scales=scales[2], activation="silu") if gated else {}
        args = sat.Mxfp4GemmArgs(rows=rows, cols=cols, width=k, out_type=kind, alpha=2.0**-8, a_codes=a, lda=k // 2, a_scales=scales[0],
                                 b_codes=b, ldb=k // 2, b_scales=scales[1], out=out, ldo=cols, **f)

        def run(call=hasty.mxfp4_gemm):
            out.zero_()
            assert call(args.address, stream()) == 0
            torch.cuda.synchronize()
            return [out]

        return run, [t.clone() for t in run(sat.lib().mxfp4_gemm)]

    near_the_limit(make, 256, 1 << 16)


@pytest.mark.parametrize("rows,hidden", [(1500, 704), (200, 200), (30, 1000)])
def test_gated_product_and_its_slopes(hasty, rows, hidden):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)

    def make(k):
        x, w = ref.rows(g, rows, k, "bf16"), ref.rows(g, 2 * hidden, k, "bf16", scale=k**-0.5)
        dh = ref.rows(g, rows, hidden, "bf16")
        h, pre = (torch.empty(rows, n * hidden, device="cuda", dtype=torch.bfloat16) for n in (1, 2))
        f = dict(rows=rows, width=k, hidden=hidden, type="bf16", activation="gelu", w_by_output=1, x=x, ldx=k, w=w, ldw=k)
        args, again = sat.FfnArgs(h=h, ldh=hidden, preact=pre, ldp=2 * hidden, **f), sat.FfnArgs(**f)
        dx = torch.empty(rows, k, device="cuda", dtype=torch.bfloat16)
        grads = sat.FfnGrads(dh=dh, lddh=hidden, dx=dx, lddx=k)
        size = sat.ffn_gated_backward_workspace(again, grads)
        grads.workspace, grads.workspace_bytes = torch.zeros(size, device="cuda", dtype=torch.uint8), size
        assert sat.ffn_gated_workspace(args) == 0
        dz = grads._keep["workspace"][:rows * 2 * hidden * 2].view(torch.bfloat16)  # [dg du], hidden a multiple of 8

        def run(lib=hasty):
            for t in (h, pre, dz):
                t.zero_()
            assert lib.ffn_gated(args.address, stream()) == 0
            assert lib.ffn_gated_backward(again.address, grads.address, stream()) == 0
            torch.cuda.synchronize()
            return [h, pre, dz]

        return run, [t.clone() for t in run(sat.lib())]

    near_the_limit(make, 64, 1 << 14)
