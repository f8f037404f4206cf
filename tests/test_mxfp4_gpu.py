"""Microscaled 4-bit matrices and their products against the definitions."""
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


def quantize(x, kind, code_pad=0):
    """(codes, scales) of x by the library."""
    n, width = x.shape
    codes = torch.full((n, -(-width // 32) * 16 + code_pad), 0xA5, device="cuda", dtype=torch.uint8)
    scales = torch.full((max(1, sat.mxfp4_scale_bytes(n, width)),), 0xA5, device="cuda", dtype=torch.uint8)
    a = sat.Mxfp4Args(rows=n, width=width, type=kind, values=x, ldv=x.stride(0), codes=codes, ldc=codes.stride(0), scales=scales)
    assert sat.mxfp4_quantize(a, stream()) == 0, sat.gemm_last_error()
    torch.cuda.synchronize()
    return codes, scales


def dequantize(codes, scales, n, width, kind, pad=0, offset=0):
    g = torch.Generator(device="cuda")
    out = ref.rows(g, n, width, kind, pad, offset).fill_(float("nan"))
    a = sat.Mxfp4Args(rows=n, width=width, type=kind, values=out, ldv=out.stride(0), codes=codes, ldc=codes.stride(0),
                      scales=scales)
    assert sat.mxfp4_dequantize(a, stream()) == 0, sat.gemm_last_error()
    torch.cuda.synchronize()
    assert bool(torch.isnan(ref.surroundings(out)).all()), "wrote outside"
    return out


def check_quantized(x, kind, code_pad=0, pad=0, offset=0):
    codes, scales = quantize(x, kind, code_pad)
    code, byte = ref.quantized(x)
    n, width = x.shape
    stored = codes[:, :code.shape[1] // 2].cpu()
    # -0 and 0 are one value: a sign bit alone says nothing.
    lo, hi = stored & 15, stored >> 4
    got = torch.stack([lo, hi], -1).flatten(1)
    assert torch.equal(torch.where(got == 8, 0, got), torch.where(code == 8, 0, code))
    assert bool((codes[:, code.shape[1] // 2:] == 0xA5).all())
    assert torch.equal(scales.cpu(), ref.tile_scales(byte, width))
    back = dequantize(codes, scales, n, width, kind, pad, offset).cpu()
    want = ref.values(code, byte)[:, :width].to(ref.TYPES[kind])
    assert torch.equal(torch.nan_to_num(back, nan=-77.0), torch.nan_to_num(want, nan=-77.0))


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,width", [(1, 1), (1, 32), (3, 31), (2, 33), (127, 128), (128, 100), (129, 129), (5, 1000),
                                     (260, 4096), (1, 16384), (1000, 72)])
def test_quantize_sizes(n, width, kind):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + width)
    x = ref.rows(g, n, width, kind)
    x[:, ::7] *= 30
    check_quantized(x, kind)


@pytest.mark.parametrize("i", range(12))
def test_quantize_strides(i):
    rng = np.random.default_rng(i)
    g = torch.Generator(device="cuda")
    g.manual_seed(i)
    kind = ("fp32", "bf16", "fp16")[i % 3]
    n, width = int(2**rng.uniform(0, 9)), int(2**rng.uniform(0, 11))
    pad, offset = int(rng.choice([0, 1, 3, 8])), int(rng.choice([0, 1, 3, 8]))
    check_quantized(ref.rows(g, n, width, kind, pad, offset), kind, int(rng.choice([0, 16, 48])), pad, offset)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
def test_rows_off_16_bytes_among_not_a_number(kind):
    """Whole 16-byte pieces are read and written around rows that start anywhere: neighbours are neither taken nor overwritten."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for rows, width, gap, offset in [(r, w, e, o) for r in (1, 2, 3, 131) for w in (1, 2, 5, 7, 9, 33, 129, 200)
                                     for e, o in ((0, 0), (0, 3), (1, 1), (2, 6), (3, 5), (8, 7), (5, 4))]:
        x = ref.rows(g, rows, width, kind, gap, offset)
        check_quantized(x, kind, pad=gap, offset=offset)


def test_every_bf16_value_in_a_block_with_each_power():
    # All finite bf16 values, each against block maxima that put it anywhere on the grid; ties included.
    v = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    for power in (-126, -100, -10, -1, 0, 1, 2, 40, 126):
        x = torch.zeros(v.numel(), 32, device="cuda", dtype=torch.bfloat16)
        x[:, 0] = 2.0**power
        x[:, 1] = v
        check_quantized(x, "bf16")


def test_ties_saturation_and_small_blocks():
    at = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.5, 6.0, 6.5, 7.0, 7.99], device="cuda")
    for power in (-126, -30, 0, 30, 124):
        x = torch.zeros(4, 64, device="cuda")
        x[0, :12], x[0, 12] = at, 4.0
        x[1, :12], x[1, 32:44] = -at, torch.nextafter(at, torch.tensor(0.0, device="cuda"))
        x[2, :12] = torch.nextafter(at, torch.tensor(9.0, device="cuda"))
        x[2, 33] = 4.0
        check_quantized(x * 2.0**power, "fp32")
    tiny = torch.zeros(2, 32, device="cuda")
    tiny[0, 0], tiny[0, 1], tiny[1, 5] = 1e-45, -3e-42, 2.0**-126
    check_quantized(tiny, "fp32")
    top = torch.full((1, 32), torch.finfo(torch.float32).max, device="cuda")
    check_quantized(top, "fp32")


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
def test_blocks_that_are_not_finite(kind):
    x = torch.ones(3, 96, device="cuda", dtype=ref.TYPES[kind])
    x[0, 3], x[1, 40], x[2, 95] = float("nan"), float("inf"), float("-inf")
    check_quantized(x, kind)


def random_matrix(g, n, width):
    """A quantised matrix with its values: any codes, scales of a few powers."""
    blocks = -(-width // 32)
    code = torch.randint(0, 16, (n, blocks * 32), device="cuda", generator=g, dtype=torch.uint8)
    code[:, width:] = 0
    byte = torch.randint(117, 128, (n, blocks), device="cuda", generator=g, dtype=torch.uint8)
    code, byte = code.cpu(), byte.cpu()
    return ref.pack(code, blocks * 16).cuda(), ref.tile_scales(byte, width).cuda(), ref.values(code, byte).cuda()


class Product:
    def __init__(self, seed, rows, cols, width, out="fp32", activation=None, alpha=1.0, pad=0, offset=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.rows, self.cols, self.width, self.out_kind, self.alpha = g, rows, cols, width, out, alpha
        self.activation, self.pad, self.offset = activation, pad, offset
        self.a, self.b = random_matrix(g, rows, width), random_matrix(g, cols, width)
        self.up = random_matrix(g, cols, width) if activation is not None else None

    def args(self, out):
        f = dict(rows=self.rows, cols=self.cols, width=self.width, out_type=self.out_kind, activation=self.activation or "none",
                 alpha=self.alpha, a_codes=self.a[0], lda=self.a[0].stride(0), a_scales=self.a[1], b_codes=self.b[0],
                 ldb=self.b[0].stride(0), b_scales=self.b[1], out=out, ldo=out.stride(0))
        if self.up is not None:
            f.update(up_codes=self.up[0], ldu=self.up[0].stride(0), up_scales=self.up[1])
        return sat.Mxfp4GemmArgs(**f)

    def run(self, to=None):
        out = ref.rows(self.g, self.rows, self.cols, self.out_kind, self.pad, self.offset).fill_(float("nan"))
        assert sat.mxfp4_gemm(self.args(out), stream() if to is None else to) == 0, sat.gemm_last_error()
        torch.cuda.synchronize()
        assert bool(torch.isnan(ref.surroundings(out)).all()), "wrote outside"
        return out

    def check(self):
        out = self.run()

        def product(b):
            # Alpha is an fp32 factor: one rounding more.
            z, size = self.alpha * (self.a[2] @ b[2].t()), abs(self.alpha) * (self.a[2].abs() @ b[2].abs().t())
            return z, ref.sum_error(self.width, size) + 2.0**-24 * z.abs()

        z, off = product(self.b)
        if self.up is not None:
            u, off_u = product(self.up)
            a, _ = ref.act(z, self.activation)
            # Activations in fp32: 2^-20, and for large arguments of exp the argument's own rounding.
            off_a = 1.13 * off + 2.0**-20 * (a.abs() + z.abs() * 2.0**-3)
            off = off_a * (u.abs() + off_u) + a.abs() * off_u + 2.0**-23 * (a * u).abs()
            z = a * u
        ref.assert_within(out, z, off + ref.half_step(z.abs() + off, self.out_kind), "out")
        return out


SIZES = [(1, 128, 256), (1, 1, 32), (1, 8, 1), (3, 333, 1000), (16, 1024, 4096), (17, 256, 520), (40, 136, 64), (64, 640, 2048),
         (65, 128, 96), (128, 128, 128), (129, 257, 385), (300, 72, 1056), (256, 512, 512), (200, 2000, 31), (1000, 136, 224)]


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,width", SIZES)
def test_product_sizes(rows, cols, width, out):
    Product(rows + cols, rows, cols, width, out).check()


@pytest.mark.parametrize("activation", ["none", "silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("rows,cols,width", SIZES)
def test_gated_product_sizes(rows, cols, width, activation):
    Product(rows + cols, rows, cols, width, "bf16" if rows % 2 else "fp32", activation, 0.125).check()


@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols,width", [(66, 40, 4100), (129, 104, 16000), (70, 300, 2080), (300, 130, 30000), (4, 300, 16000)])
def test_long_sums_of_few_outputs(rows, cols, width, out, activation, pad):
    """Tiles that several CTAs share."""
    Product(rows + cols, rows, cols, width, out, activation, 0.125, pad).check()


@pytest.mark.parametrize("activation", [None, "silu"])
def test_product_of_many_tiles(activation):
    Product(1, 2700, 4104, 1312, "bf16", activation).check()
    Product(2, 4200, 2048, 1024, "fp32", activation).check()


@pytest.mark.parametrize("i", range(16))
def test_product_strides(i):
    rng = np.random.default_rng(i)
    rows, cols, width = (int(2**rng.uniform(0, t)) for t in (10, 10, 11))
    Product(i, rows, cols, width, ("fp32", "bf16", "fp16")[i % 3], (None, "silu", None, "gelu")[i % 4], float(rng.choice([1.0, -0.7])),
            int(rng.choice([0, 1, 3, 8])), int(rng.choice([0, 1, 3, 8]))).check()


def test_ones_count():
    # Whole numbers are exact: every code and scale has to reach its place.
    for rows, cols, width in ((1, 300, 4000), (50, 300, 4000), (300, 300, 4000), (2600, 4100, 500)):
        p = Product(1, rows, cols, width)
        for m, n in ((p.a, rows), (p.b, cols)):
            code = torch.full((n, -(-width // 32) * 32), 2, dtype=torch.uint8)  # 1.0
            code[:, width:] = 0
            byte = torch.full((n, -(-width // 32)), 127, dtype=torch.uint8)
            m[0].copy_(ref.pack(code, m[0].shape[1]))
            m[1].copy_(ref.tile_scales(byte, width))
        assert bool((p.run() == width).all())


def test_scales_of_nan_stay_in_their_row_and_column():
    for rows in (5, 200):
        p = Product(3, rows, 264, 200)
        clean = p.run().clone()
        code, byte = torch.zeros(1, 224, dtype=torch.uint8), torch.full((1, 7), 127, dtype=torch.uint8)
        byte[0, 3] = 255
        one = ref.tile_scales(byte, 200).view(-1, 32, 4, 4)[:, 0, 0]
        p.a[1].view(-1, 2, 32, 4, 4)[0, :, 2, 0] = one.cuda()  # row 2
        out = p.run()
        assert bool(torch.isnan(out[2]).all())
        keep = [r for r in range(rows) if r != 2]
        assert torch.equal(out[keep], clean[keep])


def test_products_repeat_follow_the_stream_and_are_captured():
    for rows, cols, width in ((1, 1024, 8192), (200, 600, 1000), (2600, 2600, 512)):
        p = Product(4, rows, cols, width, "bf16")
        want = p.run()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        assert all(torch.equal(p.run(side.cuda_stream), want) for _ in range(3))
        out = torch.empty_like(want)
        graph, args = torch.cuda.CUDAGraph(), p.args(out)
        with torch.cuda.graph(graph):
            assert sat.mxfp4_gemm(args, stream()) == 0, sat.gemm_last_error()
        for _ in range(2):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_feed_forward_block_trained_in_16_bits_and_served_in_4():
    # The operators as they are used together: the gated product in bf16, then the same weights microscaled; each step of the
    # second against the definition on what the step before it gave.
    rows, width, hidden = 300, 256, 512
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, w = ref.rows(g, rows, width, "bf16"), ref.rows(g, 2 * hidden, width, "bf16", scale=width**-0.5)
    down = ref.rows(g, width, hidden, "bf16", scale=hidden**-0.5)
    h = torch.empty(rows, hidden, device="cuda", dtype=torch.bfloat16)
    a = sat.FfnArgs(rows=rows, width=width, hidden=hidden, type="bf16", activation="silu", w_by_output=1, x=x, ldx=width, w=w,
                    ldw=width, h=h, ldh=hidden)
    sat.check(sat.ffn_gated(a, stream()))
    y = torch.empty(rows, width, device="cuda", dtype=torch.bfloat16)
    with sat.Plan(rows, width, hidden, "bf16", trans_b=True, c_type="bf16") as plan:
        plan.run(h, down, y, 1.0, 0.0, stream())
        torch.cuda.synchronize()
    p = ref.Gated(x, w, True, hidden)
    ref.assert_within(h, *p.h("bf16", "silu"), "h")

    def stored(m):
        codes, scales = quantize(m, "bf16")
        return codes, scales, ref.values(*ref.quantized(m)).cuda()

    parts = {n: stored(m) for n, m in (("x", x), ("gate", w[:hidden]), ("up", w[hidden:]), ("down", down))}

    def gemm(n, m, k, b, up=None, left=None):
        q = Product.__new__(Product)
        q.g, q.rows, q.cols, q.width, q.out_kind, q.alpha, q.pad, q.offset = g, n, m, k, "bf16", 1.0, 0, 0
        q.activation, q.a, q.b, q.up = "silu" if up else None, left, b, up
        return q.check()

    h4 = gemm(rows, hidden, width, parts["gate"], parts["up"], parts["x"])
    y4 = gemm(rows, width, hidden, parts["down"], None, stored(h4))
    # Four bits are off by at most a quarter of a value (6 for up to 8, halfway between neighbours below): the answers agree in
    # the large. 2-norms: x, w and h off by about 0.1 of theirs each.
    off = float((y4.double() - y.double()).norm() / y.double().norm())
    assert off < 0.5


def test_offsets_past_32_bits():
    ld = (1 << 31) - 32  # bytes: rows 2 GB apart
    p = Product(5, 4, 40, 200)
    want = p.run()
    big = torch.zeros(3 * ld + 112, device="cuda", dtype=torch.uint8)
    a = big.as_strided((4, 112), (ld, 1))
    a.copy_(p.a[0])
    p.a = (a, *p.a[1:])
    assert torch.equal(p.run(), want)


def test_scales_of_every_size():
    # Scales at both ends: powers that cancel are exact, whatever they are, as long as the products are normal numbers.
    for ea, eb in ((254, 0), (0, 254), (127, 127), (200, 54), (10, 240), (3, 250), (190, 100)):
        p = Product(3, 70, 136, 256)
        for m, n, e in ((p.a, 70, ea), (p.b, 136, eb)):
            code = ref.quantized(torch.randn(n, 256, generator=torch.Generator().manual_seed(n)))[0]
            byte = torch.full((n, 8), e, dtype=torch.uint8)
            m[0].copy_(ref.pack(code, m[0].shape[1]))
            m[1].copy_(ref.tile_scales(byte, 256))
            m[2].copy_(ref.values(code, byte))
        p.check()


def test_weights_quantised_as_two_halves_of_a_buffer():
    # Strides of the gate's and the other weights may differ, and rows may lie inside a larger buffer.
    p = Product(5, 90, 200, 160, "bf16", "silu")
    wide = torch.zeros(200, 160, device="cuda", dtype=torch.uint8)
    wide[:, :80] = p.up[0]
    want = p.run().clone()
    p.up = (wide[:, :80], *p.up[1:])
    assert torch.equal(p.run(), want)
