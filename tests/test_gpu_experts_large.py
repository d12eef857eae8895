"""Routing and 4-bit products past 2^31 elements or bytes: the last rows, whose
offsets need more than 32 bits, equal those of a call that has them alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative


@pytest.fixture(scope="module", autouse=True)
def fp():
    import fp8_mixed_precision_gb300 as fp
    fp.lib()
    return fp


@pytest.mark.parametrize("how", [dict(renormalize=False), dict(score="sigmoid", groups=8, groups_kept=3, group_top=2)])
def test_logits_past_32_bits(fp, how):
    T, E, k = 2 ** 21 + 37, 1024, 6
    bias = torch.randn(E, device="cuda") * 0.1 if "groups" in how else None
    logits = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_()
    assert logits.numel() > 2 ** 31
    w, e = fp.fp8_route_fwd(logits, k, bias=bias, **how)
    dw = torch.randn((T, k), device="cuda")
    back = {n: how[n] for n in ("score", "renormalize") if n in how}
    d = fp.fp8_route_bwd(dw, logits, w, e, **back)
    for rows in (slice(0, 40), slice(T - 40, T)):
        part = logits[rows].contiguous()
        w2, e2 = fp.fp8_route_fwd(part, k, bias=bias, **how)
        assert torch.equal(e[rows], e2)
        # sums over the lanes in another order: 10 additions of a weight's sum, and its quotient
        assert bool(((w[rows] - w2).abs() <= 16 * U * w2).all())
        d2 = fp.fp8_route_bwd(dw[rows].contiguous(), part, w[rows].contiguous(), e2, **back)
        # likewise, and the rounding to bf16; a gradient may cancel down from its parts' size
        size = (w[rows] * dw[rows]).abs().sum(1, keepdim=True)
        assert bool(((d[rows].float() - d2.float()).abs() <= 2 * UB * d2.float().abs() + 32 * U * size).all())


def half_of(codes, scale, group):
    """Values in 64 bits of codes without zero points."""
    q = torch.stack((codes % 16, codes // 16), -1).flatten(-2).double() - 8.0
    return q * scale.double()[..., torch.arange(q.shape[-1], device=codes.device) // group]


def test_stack_past_32_bits_for_several_tokens(fp):
    E, K, F, N, T, k, group = 1024, 2080, 1024, 64, 6, 2, 128
    gu = fp.W4Weight(torch.randint(0, 256, (E, 2 * F, K // 2), dtype=torch.uint8, device="cuda"),
                     (torch.rand((E, 2 * F, -(-K // group)), device="cuda") * 0.02).bfloat16(), None, group)
    dn = fp.W4Weight(torch.randint(0, 256, (E, N, F // 2), dtype=torch.uint8, device="cuda"),
                     (torch.rand((E, N, F // group), device="cuda") * 0.02).bfloat16(), None, group)
    assert gu.codes.numel() > 2 ** 31
    x = torch.randn((T, K), device="cuda").bfloat16()
    e = torch.tensor([[E - 1, 0], [E - 2, E - 1], [E - 1, 5], [-1, E - 1], [E - 3, E - 2], [1, E - 1]],
                     dtype=torch.int32, device="cuda")
    w = torch.rand((T, k), device="cuda")
    y = fp.fp8_w4_experts(x, w, e, gu, dn).double()
    want, bound = torch.zeros_like(y), torch.zeros_like(y)
    for i in e.unique().tolist():
        if i < 0:
            continue
        t, j = (e == i).nonzero(as_tuple=True)
        wg, wd = half_of(gu.codes[i], gu.scale[i], group), half_of(dn.codes[i], dn.scale[i], group)
        xt = x[t].double()
        p, size = xt @ wg.t(), xt.abs() @ wg.abs().t() * (2 * K / 16 + 64) * U
        g, u = p[:, :F], p[:, F:]
        a = g * torch.sigmoid(g)
        h = a * u
        # |silu'| <= 1.13, silu within 2^-20 of the gate; h rounded to bf16
        eh = (1.13 * size[:, :F] + g.abs() * 2.0 ** -20) * (u.abs() + size[:, F:]) + a.abs() * size[:, F:]
        eh = eh * 1.01 + h.abs() * UB * 1.01
        z = h @ wd.t()
        ez = (h.abs() @ wd.abs().t()) * (2 * F / 16 + 64) * U * (1 + UB) + eh @ wd.abs().t()
        ww = w[t, j].double()[:, None]
        want.index_add_(0, t, ww * z)
        bound.index_add_(0, t, ww * (ez + z.abs() * (k + 2) * U))
    assert bool(((y - want).abs() <= bound + want.abs() * UB + 1e-38).all())


@pytest.mark.parametrize("T", [3, 20, 70])
def test_weight_past_32_bits(fp, T):
    N, K, group = 2 ** 20 + 48, 4128, 64
    w = fp.W4Weight(torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda"),
                    (torch.rand((N, -(-K // group)), device="cuda") * 0.02).bfloat16(), None, group)
    assert w.codes.numel() > 2 ** 31
    x = torch.randn((T, K), device="cuda").bfloat16()
    y = fp.fp8_w4_linear(x, w)
    for rows in (slice(0, 64), slice(N - 80, N)):
        v = half_of(w.codes[rows], w.scale[rows], group)
        want = x.double() @ v.t()
        bound = x.double().abs() @ v.abs().t() * (2 * K / 16 + 64) * U
        assert bool(((y[:, rows].double() - want).abs() <= bound + want.abs() * UB).all())
    assert fp.fp8_get_device_status() == 0
