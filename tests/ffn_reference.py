"""The feed-forward operators' definitions in 64 bits, and how far fp32
accumulation and one rounding may take an output from them.

A tensor-core instruction adds 16 products (64 of 4-bit elements) to the fp32
accumulator: each such addition is off by at most 2^-23 of the magnitudes added
so far, and its products, aligned to the largest of them, by at most 2^-23 of
it each. So a sum over K of terms whose magnitudes add up to S is off by at most
(K / 16 + 16) 2^-23 S.
"""
import math

import torch

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
FP32 = 2.0**-23


def half_step(t, kind):
    """The largest rounding of t to the type."""
    f = torch.finfo(TYPES[kind])
    return t.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def sum_error(k, magnitudes):
    return (k / 16 + 16) * FP32 * magnitudes


def act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        c = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g**3))
        return g * s, s + g * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    if kind == "relu":
        return g.clamp(min=0), (g > 0).double()
    return g, torch.ones_like(g)


def rows(g, n, width, kind, pad=0, offset=0, scale=1.0):
    """An n x width matrix of normal values whose rows are width + pad apart and start `offset` elements off a boundary."""
    whole = torch.full((offset + n * (width + pad) + 8,), float("nan"), device="cuda", dtype=TYPES[kind])
    view = whole[offset:offset + n * (width + pad)].view(n, width + pad)[:, :width]
    return view.copy_(torch.randn(n, width, device="cuda", generator=g) * scale)


def surroundings(view):
    """What lies around a matrix that `rows` made: everything in its storage but its elements."""
    whole = torch.empty(0, device="cuda", dtype=view.dtype).set_(view.untyped_storage())
    inside = torch.zeros(whole.numel(), device="cuda", dtype=torch.bool)
    inside.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    return whole[~inside]


def assert_within(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} are off, first {at}: {float(got[at])} instead of "
                             f"{float(want[at])}, at most {float(tol[at]):.3g} off")


class Gated:
    """x W of one gated product, with what rounding may do to it."""

    def __init__(self, x, w, by_output, hidden):
        self.x, w = x.double(), w.double()
        self.w = w.t() if by_output else w  # width x 2 hidden
        z, size = self.x @ self.w, self.x.abs() @ self.w.abs()
        off = sum_error(x.shape[1], size)
        self.g, self.u = z[:, :hidden], z[:, hidden:]
        self.dg, self.du = off[:, :hidden], off[:, hidden:]

    def h(self, kind, activation):
        a, slope = act(self.g, activation)
        # Derivatives are at most 1.13 (1.1 and 1.13 of silu and gelu), activations in fp32 good to 2^-20.
        h = a * self.u
        off = 1.13 * self.dg * self.u.abs() + a.abs() * self.du + 1.13 * self.dg * self.du + 2.0**-20 * (
            h.abs() + (self.g * self.u).abs() * 2.0**-3)
        return h, off + half_step(h.abs() + off, kind)


def gradients(x, w, by_output, hidden, kind, activation, dh, preact=None):
    """dx, dw and their tolerances. Of the steps: the pre-activations (exact where kept), [dg du] rounded to the type, the
    products, the last rounding (left to the caller, with the type of dw)."""
    p = Gated(x, w, by_output, hidden)
    g, u, off_g, off_u = p.g, p.u, p.dg, p.du
    if preact is not None:
        g, u = preact.double()[:, :hidden], preact.double()[:, hidden:]
        off_g = off_u = torch.zeros_like(g)
    dh = dh.double()
    a, slope = act(g, activation)
    # Second derivatives are at most 1 (0.5 of silu, 0.8 of gelu), but relu's slope jumps at 0.
    off_slope = off_g + 2.0**-20
    if activation == "relu":
        off_slope = (g.abs() <= off_g).double() + 2.0**-24
    dg, du = dh * u * slope, dh * a
    off_dg = dh.abs() * (u.abs() * off_slope + off_u * (slope.abs() + off_slope))
    off_du = dh.abs() * (1.13 * off_g + 2.0**-20 * (a.abs() + g.abs() * 2.0**-3))
    dz, off = torch.cat([dg, du], 1), torch.cat([off_dg, off_du], 1)
    off = off + half_step(dz.abs() + off, kind)
    size = dz.abs() + off
    dx, dw = dz @ p.w.t(), p.x.t() @ dz
    off_dx = off @ p.w.t().abs() + sum_error(2 * hidden, size @ p.w.t().abs())
    off_dw = p.x.t().abs() @ off + sum_error(x.shape[0], p.x.t().abs() @ size)
    if by_output:
        dw, off_dw = dw.t(), off_dw.t()
    return dx, off_dx, dw, off_dw


E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def power(n):
    return ((n + 1023) << 52).view(torch.float64)


def quantized(x):
    """(codes 0..15, scale bytes) of the rows of x, on the CPU, by the definition."""
    v = torch.nn.functional.pad(x.detach().cpu().double(), (0, -x.shape[1] % 32)).view(x.shape[0], -1, 32)
    top = v.abs().amax(-1)
    bad = ~torch.isfinite(v).all(-1)
    exponent = ((torch.where(bad, 1.0, top).view(torch.int64) >> 52) - 1023 - 2).clamp(min=-127)
    scaled = (v / power(exponent)[:, :, None]).abs()
    code = torch.zeros(v.shape, dtype=torch.uint8)
    grid = E2M1[:8]
    for c in range(1, 8):  # past the middle, or on it and the upper one even
        middle = (grid[c - 1] + grid[c]) / 2
        code += (scaled >= middle) if c % 2 == 0 else (scaled > middle)
    code = torch.where(torch.signbit(v), code + 8, code)
    code[bad] = 0
    byte = torch.where(bad, 255, exponent + 127).to(torch.uint8)
    byte[(top == 0) & ~bad] = 0
    return code.view(x.shape[0], -1), byte


def pack(code, ldc):
    out = torch.zeros(code.shape[0], ldc, dtype=torch.uint8)
    out[:, :code.shape[1] // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    return out


def tile_scales(byte, width):
    """Scale bytes (rows x blocks) in their storage order."""
    n, blocks = byte.shape
    groups = -(-width // 128)
    out = torch.zeros(-(-n // 128) * groups * 512, dtype=torch.uint8)
    r, b = torch.arange(n)[:, None], torch.arange(blocks)[None]
    out[((r // 128 * groups + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4).reshape(-1)] = byte.reshape(-1)
    return out


def values(code, byte):
    """What codes and scale bytes stand for, in 64 bits."""
    by = power(byte.long() - 127)
    by[byte == 255] = float("nan")
    return E2M1[code.long()] * by.repeat_interleave(32, 1)
