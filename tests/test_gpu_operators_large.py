"""Norm, gated feed-forward and clipping on tensors of more than 2^31 elements:
slices from both sides of that boundary equal the same rows computed alone."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _normal(shape, sigma, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, sigma, generator=g)


def test_norm(fp):
    R, C = 131072 + 1001, 16384
    x = _normal((R, C), 1.0, 1)
    w = 1 + 0.1 * _normal((C,), 1.0, 2).float()
    o = fp.fp8_rmsnorm_fwd(x, w)
    dy = _normal((R, C), 1e-2, 3)
    dx, dw = fp.fp8_rmsnorm_bwd(dy, x, o["rstd"], w)
    for a, b in ((0, 128), (131072 - 128, 131072), (131072, 131200), (131072 + 896, R)):
        p = fp.fp8_rmsnorm_fwd(x[a:b].contiguous(), w)
        assert torch.equal(o["row"][a:b], p["row"]) and torch.equal(o["rstd"][a:b], p["rstd"])
        assert torch.equal(o["row_scale_inv"][a:b], p["row_scale_inv"])
        assert torch.equal(o["col"][:, a:b], p["col"][:, :b - a])
        assert torch.equal(o["col_scale_inv"][:, a // 128], p["col_scale_inv"][:, 0])
        q, _ = fp.fp8_rmsnorm_bwd(dy[a:b].contiguous(), x[a:b].contiguous(), p["rstd"], w)
        assert torch.equal(dx[a:b], q)
    # dw: the sum of the parts' sums, within fp32 rounding of sums of this length
    parts = sum(fp.fp8_rmsnorm_bwd(dy[a:a + 16384], x[a:a + 16384], o["rstd"][a:a + 16384], w)[1].double()
                for a in range(0, R, 16384))
    assert float((dw.double() - parts).norm() / parts.norm()) < 1e-5
    assert fp.fp8_get_device_status() == 0


def test_gated(fp):
    N, K, F = 150100, 48, 14336
    x, dh = _normal((N, K), 1.0, 4), _normal((N, F), 1e-2, 5)
    w = _normal((2 * F, K), 0.2, 6)
    cache = fp.WeightCache()
    h = cache.register(w, "block")
    cache.begin_cycle()
    cache.get(h)
    y, ctx = fp.fp8_gated_fwd(x, cache, h, "block")
    dx, dw = fp.fp8_gated_bwd(dh, ctx, cache, h, "block")
    assert bool(torch.isfinite(dw.float()).all())
    for a, b in ((0, 256), (74752, 75008), (149632, 149888), (149888, N)):
        z, c = fp.fp8_gated_fwd(x[a:b].contiguous(), cache, h, "block")
        assert torch.equal(y[a:b], z)
        q, _ = fp.fp8_gated_bwd(dh[a:b].contiguous(), c, cache, h, "block")
        # the same codes; another split of the sums over 2F at this token count
        assert float((dx[a:b].double() - q.double()).norm() / q.double().norm()) < 4e-3
    assert fp.fp8_get_device_status() == 0


def test_clip(fp):
    n = 2_200_000_001
    g = [_normal((n,), 1e-2, 7), _normal((77,), 1.0, 8)]
    out = [torch.empty_like(t) for t in g]
    norm, _ = fp.GradClip(g, out).clip(1.0)
    want = math.sqrt(sum(float(p.double().square().sum()) for t in g for p in t.split(1 << 27)))
    # 67200 chunks over 304 CTAs: each thread adds up to 221 chunks' 64 squares
    # into four sums (a chain of 3600) before the fp64 joins; half of it by the root
    assert abs(float(norm) - want) < 1900 * 2.0 ** -24 * want
    coef = 1.0 / (want + 1e-6)
    for t, o in zip(g, out):
        for s in (slice(0, 1000), slice((1 << 31) - 500, (1 << 31) + 500), slice(t.numel() - 1000, None)):
            e = t[s].double() * coef
            assert bool(((o[s].double() - e).abs() <= (2.0 ** -8 + 2e-4) * e.abs() + 1e-40).all())
