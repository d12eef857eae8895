"""silu far down its negative tail.

With u = 2^-24 (fp32) and 2^-8 (bf16): |act'| / |act| <= 2 below -1, so an error
of e_G in G is 2 e_G of the result; 2e-5 for the exponential and the
reciprocal; one bf16 rounding, whose subnormals are 2^-133 apart.
"""
import pytest
import torch

import ref64 as ref

pytestmark = pytest.mark.gpu
U = ref.EPS24


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


@pytest.mark.parametrize("recipe", ["tensorwise", "block"])
@pytest.mark.parametrize("N", [5, 300])
def test_silu_far_down(fp, recipe, N):
    """Gates of -88.7 to -84: sigma is below 2^-126 in part, silu itself is a normal
    number down to there, in H and in dU = dH silu(G)."""
    K, F = 16, 128
    g = torch.Generator().manual_seed(N)
    x = torch.zeros((N, K))
    x[:, 0], x[:, 1], x[:, 2] = 1.0, torch.rand(N, generator=g), 1.0
    w = torch.zeros((2 * F, K))
    w[:F, 0], w[:F, 1], w[F:, 2] = -84.0, -4.7 * torch.rand(F, generator=g), 1.0
    x, w = x.to(torch.bfloat16).cuda(), w.to(torch.bfloat16).cuda()
    cache = fp.WeightCache()
    h = cache.register(w, recipe)
    cache.begin_cycle()
    cache.get(h)
    xq, wq = ref.operand(x.double(), recipe, "act"), ref.operand(w.double(), recipe, "weight")
    gu = xq @ wq.t()
    G, Up = gu[:, :F], gu[:, F:]
    in_range = G > -88.7  # e^-g is finite in fp32
    assert int(in_range.sum()) > F and int((G[in_range] < -87.4).sum()) > 0
    H = ref.act(G, "silu")[0] * Up
    e_g = K * U * (xq.abs() @ wq[:F].abs().t())
    for train in (False, True):
        y, ctx = fp.fp8_gated_fwd(x, cache, h, recipe, train=train)
        bad = (y.double() - H).abs() > (ref.EPS8 + 2e-5 + 2 * e_g + K * U) * H.abs() + 2.0 ** -133
        assert not bool((bad & in_range).any()), int((bad & in_range).sum())
    # dU, as the E5M2 rows that the backward pass leaves in its workspace
    dh = torch.full((N, F), 1e20, dtype=torch.bfloat16, device="cuda")
    ws = fp.gated_workspace(recipe, N, K, F, "cuda")
    fp.fp8_gated_bwd(dh, ctx, cache, h, recipe, ws=ws)
    rows = ref.decode(ws[:N * 2 * F].view(N, 2 * F)[:, F:].contiguous(), "e5m2")
    p = fp.fp8_gated_ctx_layout(recipe, ctx)
    off = p[3].value - ctx.ctx.data_ptr()
    kept = ctx.ctx[off:off + 2 * N * F].view(torch.bfloat16).view(N, F).double()
    want = dh.double() * ref.act(kept, "silu")[0]
    # by its own scale, from the largest value (57344) and E5M2's half step of 2^-3
    ratio = rows / torch.where(want == 0, torch.ones_like(want), want)
    ok = kept > -88.7
    scale = ratio[ok].median()
    assert float((ratio[ok] / scale - 1).abs().max()) <= 0.26
