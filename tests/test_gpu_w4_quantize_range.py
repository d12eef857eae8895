"""The 4-bit quantizer's scales and zero points at both ends of bf16's range, as they are defined."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def defined(w, group, zero):
    """scale, zero, codes of finite weights [N, K]: scales rounded from exact quotients, codes from fp32 ones."""
    N, K = w.shape
    p = w.float().view(N, K // group, group)
    hi, lo = p.amax(-1).clamp(min=0), p.amin(-1).clamp(max=0)
    # (the sum and the quotient rounded to fp32 each, as for numbers within its range)
    q = (((hi.double() - lo) / 2).float().double() / 7.5 if zero else torch.maximum(hi, -lo).double() / 7).float()
    s = q.bfloat16().float()
    s = torch.where(s == 0, torch.ones_like(s), s)
    z = (-lo / s).round().clamp(0, 15) if zero else torch.full_like(s, 8.0)
    c = ((p / s[..., None]).round() + z[..., None]).clamp(0, 15).view(N, K).to(torch.uint8)
    return s, z, c[:, 0::2] | c[:, 1::2] << 4


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
def test_ends_of_the_range(group, zero):
    import fp8_mixed_precision_gb300 as fp
    top = torch.finfo(torch.bfloat16).max
    g = torch.Generator().manual_seed(group)
    w = (2 * torch.rand((48, 256), generator=g) - 1) * 3e38   # hi - lo past fp32's range in every group
    w[1] = w[1].abs()
    w[2] = -w[2].abs()
    w[3, ::2], w[3, 1::2] = top, -top
    w[4] = top
    w[5] = w[5] / 2                                           # not past it
    w[6] = w[6] * 2.0 ** -120
    w = w.bfloat16()
    q = fp.fp8_w4_quantize(w.cuda(), group, zero)
    s, z, codes = defined(w, group, zero)
    assert torch.equal(q.scale.cpu().float(), s) and bool(q.scale.isfinite().all())
    assert torch.equal(q.codes.cpu(), codes)
    if zero:
        assert torch.equal(q.zero.cpu().float(), z)
    # within half a step, or a whole one where the rounded zero point cuts the end off, and the scale's rounding
    v = codes_of(q, group)
    off = (v - w.double()).abs().view(48, -1, group)
    assert bool((off <= s.double()[..., None] * 1.1).all())


def codes_of(q, group):
    c = q.codes.cpu()
    n = torch.stack((c & 15, c >> 4), -1).flatten(-2).double()
    z = 8.0 if q.zero is None else q.zero.cpu().double().repeat_interleave(group, -1)
    return (n - z) * q.scale.cpu().double().repeat_interleave(group, -1)
