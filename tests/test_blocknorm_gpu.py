"""Block norm and its gradients against the formulas in 64 bits.

Tolerances: an output is rounded once to its type (half a unit in the last
place), after fp32 arithmetic whose relative error per step is 2^-24. A value
goes through at most about a dozen such steps beside sums over a row, which
are at most 32 sequential additions in a thread and 9 across threads; so it is
within 64 x 2^-24 = 4e-6 of the sum of the sizes of what it is made of. Sums
over rows add at most 100 sequential additions at the sizes tested: 1e-5 more.
"""
import numpy as np
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import lm_reference as ref
from tests.gpu_util import stream

pytestmark = pytest.mark.gpu

EPS = 1e-5
STEP = 4e-6
KINDS = ("none", "rms", "layer")


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


class Case:
    """Inputs on the device, as the kernels see them, and in 64 bits."""

    def __init__(self, seed, rows, width, block="fp32", stream_type="fp32", post="rms", pre="rms", rows_per_gate=0,
                 gate_type=None, pad=0, offset=0, betas=True, gammas=True, residual_scale=1.0, branch_scale=1.0, shift=0.0):
        rng = np.random.default_rng(seed)
        self.rows, self.width, self.block, self.stream, self.pad, self.offset = rows, width, block, stream_type, pad, offset
        self.gate_type = gate_type or block
        self.p = {"post": post, "pre": pre, "eps": EPS, "residual_scale": residual_scale, "branch_scale": branch_scale}
        self.x, _ = ref.place(rng.standard_normal((rows, width)) + shift, stream_type, pad, offset)
        self.y, _ = ref.place(rng.standard_normal((rows, width)) * 2 + shift, block, pad, offset)
        self.w = {}
        for at, kind in (("post", post), ("pre", pre)):
            if kind != "none" and gammas:
                self.w[at + "_gamma"] = torch.from_numpy(1 + 0.2 * rng.standard_normal(width)).float().cuda()
            if kind == "layer" and betas:
                self.w[at + "_beta"] = torch.from_numpy(0.3 * rng.standard_normal(width)).float().cuda()
        self.p.update({n: ref.f64(t) for n, t in self.w.items()})
        self.gate, self.rows_per_gate, self.gate64 = None, rows_per_gate, 1.0
        if rows_per_gate:
            self.groups = -(-rows // rows_per_gate)
            self.gate, _ = ref.place(rng.standard_normal((self.groups, width)), self.gate_type, pad, offset)
            self.gate64 = np.repeat(ref.f64(self.gate), min(rows_per_gate, rows), 0)[:rows]
        self.rng = rng

    def args(self, **more):
        f = dict(rows=self.rows, width=self.width, block_type=self.block, stream_type=self.stream, gate_type=self.gate_type,
                 post_norm=self.p["post"], pre_norm=self.p["pre"], post_eps=EPS, pre_eps=EPS,
                 residual_scale=self.p["residual_scale"], branch_scale=self.p["branch_scale"], x=self.x, ldx=self.x.stride(0),
                 y=self.y, ldy=self.y.stride(0), gate=self.gate, ldg=self.gate.stride(0) if self.gate is not None else 0,
                 rows_per_gate=self.rows_per_gate, **self.w)
        return sat.BlockNormArgs(**{**f, **more})

    def forward(self, check=True):
        rows, width = self.rows, self.width
        h, wh = ref.place(np.zeros((rows, width)), self.stream, self.pad, self.offset, -77.0)
        z, wz = ref.place(np.zeros((rows, width)), self.block, self.pad, self.offset, -77.0)
        stats = {at: torch.full((rows, 2), float("nan"), device="cuda") for at in ("post", "pre") if self.p[at] != "none"}
        args = self.args(h=h, ldh=h.stride(0), z=z if self.p["pre"] != "none" else None, ldz=z.stride(0),
                         post_stats=stats.get("post"), pre_stats=stats.get("pre"))
        assert sat.rowop_block_norm(args, stream()) == 0, sat.gemm_last_error()
        torch.cuda.synchronize()
        if check:
            want = ref.block_norm(ref.f64(self.x), ref.f64(self.y), self.gate64, self.p)
            size = self.sizes(want)
            ref.assert_within(ref.f64(h), want["h"], STEP * size["h"] + ref.rounding(self.stream, want["h"]), "h")
            assert ref.sentinel_intact(h, wh, -77.0)
            if self.p["pre"] != "none":
                ref.assert_within(ref.f64(z), want["z"], STEP * size["z"] + ref.rounding(self.block, want["z"]), "z")
                assert ref.sentinel_intact(z, wz, -77.0)
            for at, got in stats.items():
                mean, r = want[at]
                ref.assert_within(ref.f64(got[:, 1:]), r, (STEP + STEP * size[at]) * r, at + " deviation")
                ref.assert_within(ref.f64(got[:, :1]), mean, STEP * size[at + " mean"], at + " mean")
        return h, z, stats

    def sizes(self, want):
        x, y, p = np.abs(ref.f64(self.x)), np.abs(ref.f64(self.y)), self.p
        size, n = {}, y
        if p["post"] != "none":
            mean, r = want["post"]
            size["post mean"] = y.mean(1, keepdims=True)
            size["post"] = y.mean(1, keepdims=True) * r
            n = (y + size["post mean"]) * r * np.abs(p.get("post_gamma", 1.0)) + np.abs(p.get("post_beta", 0.0))
        h = abs(p["residual_scale"]) * x + abs(p["branch_scale"]) * np.abs(self.gate64) * n
        size["h"] = h
        if p["pre"] != "none":
            mean, r = want["pre"]
            size["pre mean"] = h.mean(1, keepdims=True)
            size["pre"] = h.mean(1, keepdims=True) * r
            # An error of a row's h is also one of its mean and its deviation.
            size["z"] = (2 * h + size["pre mean"]) * r * np.abs(p.get("pre_gamma", 1.0)) * (1 + size["pre"]) + \
                np.abs(p.get("pre_beta", 0.0))
        return size

    def backward(self, check=True, want=("dx", "dy", "gate", "post_gamma", "post_beta", "pre_gamma", "pre_beta"), with_dh=True,
                 in_place=False):
        rows, width, p = self.rows, self.width, self.p
        h, _ = ref.place(self.rng.standard_normal((rows, width)), self.stream, self.pad, self.offset)
        dh, _ = ref.place(self.rng.standard_normal((rows, width)), self.stream, self.pad, self.offset)
        dz, _ = ref.place(self.rng.standard_normal((rows, width)), self.block, self.pad, self.offset)
        dh64, dz64 = ref.f64(dh) if with_dh else np.zeros((rows, width)), ref.f64(dz)
        stats, stats64 = {}, {}
        for at, v in (("post", self.y), ("pre", h)):
            stats64[at] = None
            if p[at] != "none":
                _, mean, r = ref.norm(ref.f64(v), p[at], None, None, EPS)
                stats[at] = torch.from_numpy(np.concatenate([mean, r], 1)).float().cuda()
                stats64[at] = (ref.f64(stats[at][:, :1]), ref.f64(stats[at][:, 1:]))
        dx, wx = (dh, None) if in_place else ref.place(np.zeros((rows, width)), self.stream, self.pad, self.offset, -77.0)
        dy, wy = (dz, None) if in_place else ref.place(np.zeros((rows, width)), self.block, self.pad, self.offset, -77.0)
        out = {"dx": dx, "dy": dy}
        names = [n for n in want if n in self.w] + (["gate"] if self.gate is not None and "gate" in want else [])
        for n in names:
            if n == "gate":
                out[n], _ = ref.place(np.zeros((self.groups, width)), self.gate_type, self.pad, self.offset)
            else:
                out[n] = torch.full((width,), float("nan"), device="cuda")
        args = self.args(h=h, ldh=h.stride(0), post_stats=stats.get("post"), pre_stats=stats.get("pre"))
        size = sat.rowop_block_norm_workspace(args)
        scratch = torch.full((size + 64,), 0x7f, device="cuda", dtype=torch.uint8)
        grads = sat.BlockNormGrads(
            dh=dh if with_dh else None, lddh=dh.stride(0), dz=dz if p["pre"] != "none" else None, lddz=dz.stride(0),
            dx=dx if "dx" in want else None, lddx=dx.stride(0), dy=dy if "dy" in want else None, lddy=dy.stride(0),
            dgate=out.get("gate"), lddg=out["gate"].stride(0) if "gate" in out else 0, workspace=scratch, workspace_bytes=size,
            **{"d" + n: out[n] for n in names if n != "gate"})
        assert sat.rowop_block_norm_backward(args, grads, stream()) == 0, sat.gemm_last_error()
        torch.cuda.synchronize()
        assert bool((scratch[size:] == 0x7f).all())
        out = {n: t for n, t in out.items() if n in want}
        if check:
            good, sizes = ref.block_norm_backward(ref.f64(self.y), ref.f64(h), dh64, dz64, self.gate64, p, stats64["post"],
                                                  stats64["pre"])
            for n, t in out.items():
                g, s, tol = good[n], sizes[n], 2 * STEP
                if n == "gate":
                    at = np.arange(0, rows, min(self.rows_per_gate, rows))
                    g, s = np.add.reduceat(g, at, 0), np.add.reduceat(s, at, 0)
                if n not in ("dx", "dy"):
                    tol += 1e-5
                dtype = {"dx": self.stream, "dy": self.block, "gate": self.gate_type}.get(n, "fp32")
                ref.assert_within(ref.f64(t), g, tol * s + ref.rounding(dtype, g), n)
            if not in_place:
                assert "dx" not in want or ref.sentinel_intact(dx, wx, -77.0)
                assert "dy" not in want or ref.sentinel_intact(dy, wy, -77.0)
        return out


WIDTHS = [1, 2, 7, 8, 31, 64, 255, 256, 257, 264, 1000, 1024, 1025, 2048, 2056, 4095, 4096, 4097, 4104, 8191, 8192, 8200,
          12289, 16384]


@pytest.mark.parametrize("block,stream_type", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("width", WIDTHS)
def test_every_width_forward_and_backward(width, block, stream_type):
    i = WIDTHS.index(width)
    rows = [1, 3, 6, 13][i % 4]
    c = Case(width, rows, width, block, stream_type, KINDS[1 + i % 2], KINDS[1 + (i // 2) % 2], [0, rows, 1, 2][i % 4],
             residual_scale=1.25, branch_scale=0.5)
    c.forward()
    c.backward()


@pytest.mark.parametrize("post", KINDS)
@pytest.mark.parametrize("pre", KINDS)
@pytest.mark.parametrize("rows_per_gate", [0, 1, 3, 10 ** 9])
def test_norms_and_gates(post, pre, rows_per_gate):
    c = Case(5, 37, 320, "fp16", "fp32", post, pre, rows_per_gate, "fp32" if rows_per_gate == 3 else "fp16")
    c.forward()
    c.backward()


@pytest.mark.parametrize("i", range(48))
def test_random_rows_strides_and_offsets(i):
    rng = np.random.default_rng(900 + i)
    block = ("bf16", "fp16", "fp32")[i % 3]
    width = int(2 ** rng.uniform(0, 13.5))
    rows = int(rng.integers(1, 1 + min(900, 400000 // width)))
    c = Case(i, rows, width, block, rng.choice([block, "fp32"]), rng.choice(KINDS), rng.choice(KINDS),
             int(rng.choice([0, 1, 2, 7, max(1, rows // 3), rows, 2 * rows])), rng.choice([block, "fp32"]),
             pad=int(rng.choice([0, 1, 3, 8])), offset=int(rng.choice([0, 1, 8])), betas=bool(rng.integers(2)),
             gammas=bool(rng.integers(2)), branch_scale=-0.75)
    c.forward()
    c.backward()


@pytest.mark.parametrize("rows,rows_per_gate", [(1300, 1300), (1300, 1), (1300, 4), (3000, 7), (700, 350), (2500, 26)])
@pytest.mark.parametrize("width", [100, 520, 1544, 2504])
def test_many_rows_share_parts_and_gates(rows, rows_per_gate, width):
    # More rows, or gate rows, than parts of the backward pass: gradients written by whole groups, by pieces, and both.
    c = Case(rows, rows, width, "bf16", "bf16", "layer", "rms", rows_per_gate, "fp32")
    c.backward()


@pytest.mark.parametrize("width,pad", [(700, 0), (1032, 8), (1537, 0), (4096, 0), (5001, 3), (8192, 0), (12290, 1), (16384, 0)])
@pytest.mark.parametrize("block,stream_type", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_many_rows_through_the_ring(width, pad, block, stream_type):
    # More rows than eight an SM: CTAs, or pairs of them, that stay for several, with the weights kept on chip or not.
    i = width % 3
    c = Case(width, 1219, width, block, stream_type, KINDS[i], KINDS[1 + i % 2], [0, 1219, 40][i], pad=pad, residual_scale=1.25)
    c.forward()
    if width in (1537, 8192):
        c.backward()


@pytest.mark.parametrize("width", [2500, 4000, 5001, 8192, 12000])
def test_many_rows_give_the_same_bits_every_time(width):
    # Rings whose stages are no multiple of the groups that share them: a stage goes from group to group.
    c = Case(3, 2049, width, "fp32", "fp32", "none", "layer", 2049)
    h, z, _ = c.forward()
    for _ in range(60):
        again = c.forward(check=False)
        assert torch.equal(h, again[0]) and torch.equal(z, again[1])


@pytest.mark.parametrize("width", [96, 1000, 2001, 6000, 16384])
def test_rows_far_from_zero_keep_their_variance(width):
    # Mean 300, deviation 1: a variance from the difference of two sums would be lost to rounding.
    Case(3, 5, width, "fp32", "fp32", "layer", "layer", shift=300.0).forward()


@pytest.mark.parametrize("width", [40, 513, 4096, 9000])
def test_subsets_of_gradients_and_no_dh(width):
    for want in (("dx",), ("dy",), ("gate",), ("pre_gamma", "post_gamma"), ("post_beta",)):
        Case(8, 11, width, "bf16", "fp32", "layer", "layer", 4).backward(want=want, with_dh=False)


@pytest.mark.parametrize("width,pad", [(96, 0), (1000, 3), (4096, 0), (8192, 8), (16384, 0)])
def test_in_place(width, pad):
    a, b = (Case(4, 9, width, "bf16", "bf16", "rms", "layer", 9, pad=pad) for _ in range(2))
    h, z, _ = a.forward()
    args = b.args(h=b.x, ldh=b.x.stride(0), z=b.y, ldz=b.y.stride(0))
    assert sat.rowop_block_norm(args, stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(b.x, h) and torch.equal(b.y, z)
    one = Case(4, 9, width, "bf16", "bf16", "rms", "layer", 9, pad=pad).backward()
    two = Case(4, 9, width, "bf16", "bf16", "rms", "layer", 9, pad=pad).backward(in_place=True)
    assert all(torch.equal(one[n], two[n]) for n in one)


@pytest.mark.parametrize("width", [24, 1537, 4096, 10000])
def test_results_repeat_and_rows_do_not_depend_on_one_another(width):
    c = Case(12, 300, width, "fp16", "fp32", "layer", "rms", 100)
    first = [t.clone() for t in (*c.forward()[:2], )]
    for _ in range(3):
        assert all(torch.equal(s, t) for s, t in zip(first, c.forward(check=False)[:2]))
    state = c.rng.bit_generator.state
    grads = c.backward(check=False)
    for _ in range(3):
        c.rng.bit_generator.state = state
        again = c.backward(check=False)
        assert all(torch.equal(grads[n], again[n]) for n in grads)
    # A NaN and an infinity stay in their rows.
    c.y[7, width // 2] = float("nan")
    c.x[8, 0] = float("inf")
    got = c.forward(check=False)[:2]
    keep = [r for r in range(300) if r not in (7, 8)]
    assert all(torch.equal(s[keep], t[keep]) for s, t in zip(first, got))
    assert bool(got[0][7].isnan().any()) and bool(got[0][8].isinf().any())


def test_constant_and_zero_rows():
    c = Case(1, 4, 1000, "fp32", "fp32", "layer", "rms")
    c.y[0] = 3.5
    c.y[1] = 0.0
    c.x[1] = 0.0
    c.forward()
    one = Case(1, 5, 1, "fp32", "fp32", "layer", "layer")  # a row of one element is its own mean
    one.forward()
    one.backward()


def test_no_rows_set_the_weights_gradients_to_zero():
    g = torch.full((4, 24), float("nan"), device="cuda")
    args = sat.BlockNormArgs(rows=0, width=24, post_norm="layer", pre_norm="layer")
    grads = sat.BlockNormGrads(dpost_gamma=g[0], dpost_beta=g[1], dpre_gamma=g[2], dpre_beta=g[3])
    assert sat.rowop_block_norm_backward(args, grads, stream()) == 0, sat.gemm_last_error()
    torch.cuda.synchronize()
    assert bool((g == 0).all())


def test_offsets_past_32_bits():
    ld, rows, width = 1 << 27, 18, 520
    big = [torch.empty((rows - 1) * ld + width, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    views = [t.as_strided((rows, width), (ld, 1)) for t in big]
    c = Case(2, rows, width, "bf16", "bf16", "rms", "rms")
    views[0].copy_(c.x)
    views[1].copy_(c.y)
    h, z, _ = c.forward()
    args = c.args(x=views[0], ldx=ld, y=views[1], ldy=ld, h=views[0], ldh=ld, z=views[1], ldz=ld)
    assert sat.rowop_block_norm(args, stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(views[0], h) and torch.equal(views[1], z)


def test_on_another_stream():
    c = Case(2, 64, 2048, "bf16", "fp32", "rms", "rms")
    h, z, _ = c.forward()
    side = torch.cuda.Stream()
    h2, z2 = torch.empty_like(h), torch.empty_like(z)
    side.wait_stream(torch.cuda.current_stream())
    args = c.args(h=h2, ldh=h2.stride(0), z=z2, ldz=z2.stride(0))
    assert sat.rowop_block_norm(args, side.cuda_stream) == 0
    side.synchronize()
    assert torch.equal(h, h2) and torch.equal(z, z2)


@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms"), ("none", "layer"), ("rms", "none")])
def test_gradients_against_differences(post, pre):
    # The forward formulas in 64 bits, moved along a random direction of all inputs at once, against the
    # gradients' product with it. Central differences of step 1e-4 are within about 1e-7 of the derivative.
    rows, width, step = 6, 40, 1e-4
    c = Case(21, rows, width, "fp32", "fp32", post, pre, 2)
    x, y, gate = ref.f64(c.x), ref.f64(c.y), ref.f64(c.gate)
    rng = np.random.default_rng(3)
    dh, dz = rng.standard_normal((2, rows, width)).astype(np.float32)
    move = {n: rng.standard_normal(v.shape) for n, v in {"x": x, "y": y, "gate": gate, **{n: ref.f64(t) for n, t in c.w.items()}}.items()}

    def value(t):
        p = {**c.p, **{n: c.p[n] + t * move[n] for n in c.w}}
        o = ref.block_norm(x + t * move["x"], y + t * move["y"], np.repeat(gate + t * move["gate"], 2, 0), p)
        return (dh * o["h"]).sum() + (0 if pre == "none" else (dz * o["z"]).sum())

    slope = (value(step) - value(-step)) / (2 * step)
    h, _, stats = c.forward()
    got = {n: torch.empty(t.shape, device="cuda") for n, t in {"x": c.x, "y": c.y, "gate": c.gate, **c.w}.items()}
    args = c.args(h=h, ldh=h.stride(0), post_stats=stats.get("post"), pre_stats=stats.get("pre"))
    size = sat.rowop_block_norm_workspace(args)
    scratch = torch.empty(max(size, 1), device="cuda", dtype=torch.uint8)
    grads = sat.BlockNormGrads(
        dh=torch.from_numpy(dh).cuda(), lddh=width, dz=torch.from_numpy(dz).cuda() if pre != "none" else None, lddz=width,
        dx=got["x"], lddx=width, dy=got["y"], lddy=width, dgate=got["gate"], lddg=width, workspace=scratch,
        workspace_bytes=size, **{"d" + n: got[n] for n in c.w})
    assert sat.rowop_block_norm_backward(args, grads, stream()) == 0, sat.gemm_last_error()
    torch.cuda.synchronize()
    terms = np.concatenate([(ref.f64(got[n]) * move[n]).ravel() for n in got])
    assert abs(terms.sum() - slope) <= 2e-5 * np.abs(terms).sum()
