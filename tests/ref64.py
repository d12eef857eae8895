"""Plain 64-bit statements of the norm, the gated feed-forward and the FP8
rounding they use, for the GPU tests (float64 torch on whatever device the
inputs are on; no code of the library)."""
import math

import torch

FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS24 = 2.0 ** -24  # unit roundoff of fp32
EPS8 = 2.0 ** -8    # unit roundoff of bf16 (8 significand bits)


def f32(v):
    return v.to(torch.float32).to(torch.float64)


def round_fp8(v, fmt):
    """Saturating round-to-nearest-even onto the FP8 format's values."""
    mant, emin = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.frexp(v)[1].to(torch.float64) - 1.0
    step = torch.exp2(torch.clamp(e, min=emin) - mant)
    return torch.clamp(torch.round(v / step) * step, -FMAX[fmt], FMAX[fmt])


def decode(b, fmt):
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    return b.view(dt).to(torch.float32).to(torch.float64)


def scale_of(amax, fmt):
    """fp32(fmax / amax), 1 for an empty or all-zero group, and its fp32 reciprocal."""
    one = torch.ones_like(amax)
    s = f32(torch.where(amax > 0, FMAX[fmt] / torch.where(amax > 0, amax, one), one))
    s = torch.clamp(s, max=torch.finfo(torch.float32).max)
    return s, f32(1.0 / s)


def blocks(v, fmt, a=1, b=128):
    """(values on the FP8 grid, scale, scale_inv) of a x b blocks of v [R, C]."""
    R, C = v.shape
    A, B = -(-R // a), -(-C // b)
    p = torch.zeros((A * a, B * b), dtype=torch.float64, device=v.device)
    p[:R, :C] = v
    p = p.view(A, a, B, b)
    s, si = scale_of(p.abs().amax((1, 3)), fmt)
    q = round_fp8(f32(f32(p) * s[:, None, :, None]), fmt)
    return q.view(A * a, B * b)[:R, :C], s, si


def block_values(v, fmt, a=1, b=128):
    q, _, si = blocks(v, fmt, a, b)
    return q * si.repeat_interleave(a, 0).repeat_interleave(b, 1)[:v.shape[0], :v.shape[1]]


def tensor_values(v, fmt):
    s, si = scale_of(v.abs().amax(), fmt)
    return round_fp8(f32(f32(v) * s), fmt) * si


def operand(v, recipe, role):
    """What the FP8 operand made of v stands for (rowwise layout)."""
    fmt = "e5m2" if role == "grad" else "e4m3"
    if recipe != "block":
        return tensor_values(v, fmt)
    return block_values(v, fmt, 128, 128) if role == "weight" else block_values(v, fmt)


def act(g, name):
    """act(g) and act'(g)."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    phi = torch.special.erfc(-g / math.sqrt(2)) / 2
    return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
