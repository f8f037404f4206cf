"""The activations' relative accuracy, in the tails too, where an activation is
itself small: every 16-bit gate, and fp32 outputs of exact gates.

Roundings are counted in 2^-24 of a value (fp32's half step):
- GELU: the fit of the tail 0.4, t 3 (its reciprocal 2, its sum one), which the Mills ratio passes on at most once, eight
  steps of the polynomial 3 (each counts by its share of the sum; evaluated in fp32 against 64 bits), the density 12 (two
  powers of two 4 each, the constant and three products), three more products and that with u: 23.
- SiLU, g e / (1 + e) with e = exp(-|g|): exp 10 (two powers of two 4 each, two products), 1 + e one, its reciprocal 2, three
  products: 16.
- GELU by tanh: as SiLU, and 6 of the argument of exp (constants, squares, products), which exp takes to 6 times the
  argument's size.
Outputs of 16 bits: the argument of exp is a rounded product with a constant that is off by 1.33e-8 (of the argument, 0.22
half steps), so exp is off by 1.25 half steps times its size besides; GELU's argument g^2 / 2 has the rounding of the square
too, 2.25 (GELU by tanh: within the 8 that are counted below). Against outputs that are rounded to 2^-9 or 2^-12 that is little.
So 2^-19 (32 of them) and, by tanh, 2^-21 times the argument. Below fp32's normal numbers a rounding is up to 2^-149.
"""
import math

import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests import ffn_reference as ref
from tests.gpu_util import stream

pytestmark = pytest.mark.gpu

KINDS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


def argument(g):
    """What exp gets in GELU by tanh."""
    return 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g**3).abs()


def tolerance(g, kind, fine=False):
    """Relative, of the activation. fine: for fp32 outputs."""
    if kind in ("none", "relu"):
        return torch.full_like(g, 2.0**-24)
    coarse = {"silu": 1.25 * g.abs().clamp(max=150.0), "gelu": 2.25 * (g * g / 2).clamp(max=128.0), "gelu_tanh": torch.zeros_like(g)}[kind]
    return 2.0**-19 + (2.0**-21 * argument(g).clamp(max=200.0) if kind == "gelu_tanh" else 0.0) + (0.0 if fine else 2.0**-24 * coarse)


def tiny(g):
    """The absolute error of a factor below the normal numbers times the gate."""
    return 2.0**-147 * (1 + g.abs())


def exact_gates(lowest):
    """All multiples of 2^lowest with 12 bits and a sign, as digits of three bits in four blocks of 32 columns, of one scale
    each: any sum of them is exact. A fifth block holds the 1 of the other factor."""
    n = torch.arange(-4095, 4096)
    code = torch.zeros(n.numel(), 160, dtype=torch.uint8)
    for block in range(4):
        for bit in range(3):
            one = (n.abs() >> (3 * block + bit)) & 1
            code[:, 32 * block + bit] = torch.where(one > 0, torch.tensor([2, 4, 6])[bit] + 8 * (n < 0), 0)  # 1, 2, 4
    code[:, 128] = 2
    gate, up = torch.zeros(1, 160, dtype=torch.uint8), torch.zeros(1, 160, dtype=torch.uint8)
    gate[0, :128] = 2
    up[0, 128] = 2
    byte = torch.tensor([127 + lowest + 3 * b for b in range(4)] + [127], dtype=torch.uint8)[None]
    return n.double().cuda() * 2.0**lowest, code, gate, up, byte


@pytest.mark.parametrize("kind", KINDS[1:])
@pytest.mark.parametrize("lowest", [-5, -8, -14])
@pytest.mark.parametrize("rows", [50, 8191])
def test_fp32_outputs_of_exact_gates(kind, lowest, rows):
    g, code, gate, up, byte = exact_gates(lowest)
    cols = 5

    def stored(c, b):
        return ref.pack(c, 80).cuda(), ref.tile_scales(b.expand(c.shape[0], 5), 160).cuda()

    (bc, bs), (uc, us) = (stored(m.expand(cols, 160), torch.full((1, 5), 127, dtype=torch.uint8)) for m in (gate, up))
    for first in range(0, g.numel(), 50 * 16 if rows == 50 else rows):
        n = min(rows, g.numel() - first)
        ac, as_ = stored(code[first:first + n], byte)
        out = torch.full((n, cols), float("nan"), device="cuda")
        args = sat.Mxfp4GemmArgs(rows=n, cols=cols, width=160, out_type="fp32", activation=kind, alpha=1.0, a_codes=ac, lda=80,
                                 a_scales=as_, b_codes=bc, ldb=80, b_scales=bs, up_codes=uc, ldu=80, up_scales=us, out=out, ldo=cols)
        assert sat.mxfp4_gemm(args, stream()) == 0, sat.gemm_last_error()
        torch.cuda.synchronize()
        x = g[first:first + n, None].expand(n, cols)
        want = ref.act(x, kind)[0]
        ref.assert_within(out, want, want.abs() * tolerance(x, kind, fine=True) + tiny(x), f"{kind} of {float(x[0, 0])} ..")


def gates(kind):
    """Every finite value that is normal in fp32 (what products make of others is not looked at here)."""
    v = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(ref.TYPES[kind])
    return v[torch.isfinite(v) & (v.float().abs() >= 2.0**-126)]


@pytest.mark.parametrize("activation", KINDS)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_every_gate(kind, activation):
    """x = (g, 1) and weights that pick them: the gate and a factor of 1, exactly."""
    g = gates(kind)
    n = g.numel()
    x = torch.zeros(n, 8, device="cuda", dtype=g.dtype)
    x[:, 0], x[:, 1] = g, 1
    w = torch.zeros(2, 8, device="cuda", dtype=g.dtype)
    w[0, 0], w[1, 1] = 1, 1
    for rows in (n, 64):
        h = torch.full((rows, 1), float("nan"), device="cuda", dtype=g.dtype)
        at = torch.randperm(n, generator=torch.Generator().manual_seed(1))[:rows].cuda() if rows < n else torch.arange(n, device="cuda")
        xs = x[at].contiguous()
        args = sat.FfnArgs(rows=rows, width=8, hidden=1, type=kind, activation=activation, w_by_output=1, x=xs, ldx=8, w=w, ldw=8,
                           h=h, ldh=1)
        assert sat.ffn_gated_workspace(args) == 0
        assert sat.ffn_gated(args, stream()) == 0, sat.gemm_last_error()
        torch.cuda.synchronize()
        v = g[at].double()
        want = ref.act(v, activation)[0]
        off = want.abs() * tolerance(v, activation) + tiny(v)
        ref.assert_within(h[:, 0], want, off + ref.half_step(want.abs() + off, kind), "h")


def slope_terms(g, kind):
    """The derivative and the magnitude of what it is the sum of."""
    d = ref.act(g, kind)[1]
    if kind == "silu":
        s = torch.sigmoid(g)
        return d, s + (g * s * torch.sigmoid(-g)).abs()
    if kind == "gelu":
        c = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return d, c + (g * torch.exp(-g * g / 2)).abs() / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        y = math.sqrt(2 / math.pi) * (g + 0.044715 * g**3)
        s, r = torch.sigmoid(2 * y), torch.sigmoid(-2 * y)
        return s + g * s * r * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g), s + (
            g * s * r * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)).abs()
    return d, d.abs()


@pytest.mark.parametrize("recompute", [False, True])
@pytest.mark.parametrize("activation", KINDS)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_slopes_of_every_gate(kind, activation, recompute):
    """Gradients of the same: dx = (dh a'(g), dh a(g)) with dh = u = 1, exactly dg and du (from 2^-126 on, as above)."""
    g = gates(kind)
    n = g.numel()
    x = torch.zeros(n, 8, device="cuda", dtype=g.dtype)
    x[:, 0], x[:, 1] = g, 1
    w = torch.zeros(2, 8, device="cuda", dtype=g.dtype)
    w[0, 0], w[1, 1] = 1, 1
    pre, dh, dx = x[:, :2].contiguous(), torch.ones(n, 8, device="cuda", dtype=g.dtype), torch.full_like(x, float("nan"))
    args = sat.FfnArgs(rows=n, width=8, hidden=1, type=kind, activation=activation, w_by_output=1, x=x, ldx=8, w=w, ldw=8,
                       **({} if recompute else dict(preact=pre, ldp=2)))
    grads = sat.FfnGrads(dh=dh, lddh=8, dx=dx, lddx=8)
    size = sat.ffn_gated_backward_workspace(args, grads)
    grads.workspace, grads.workspace_bytes = torch.empty(size, device="cuda", dtype=torch.uint8), size
    assert sat.ffn_gated_backward(args, grads, stream()) == 0, sat.gemm_last_error()
    torch.cuda.synchronize()
    v = g.double()
    want, size = slope_terms(v, activation)
    off = size * tolerance(v, activation) + tiny(v) + 2.0**-126
    ref.assert_within(dx[:, 0], want, off + ref.half_step(want.abs() + off, kind), "dg")
    a = ref.act(v, activation)[0]
    off = a.abs() * tolerance(v, activation) + tiny(v) + 2.0**-126
    ref.assert_within(dx[:, 1], a, off + ref.half_step(a.abs() + off, kind), "du")
    assert not bool(dx[:, 2:].any())
