"""Gradients of the gated feed-forward row by row and column by column: a wrong
last row, column or group of 16 tokens of a large tensor cannot hide in the
norm of the whole.

An output sums at least 128 products.  A code of dG or dU on the other side of a
tie (1.7e-5 of them with GELU, fewer with silu) moves one term by a quarter of
its value at most: of a term five times the root mean square, 5 / 4 / sqrt(128)
= 0.11 of the row's or column's norm, so 0.125 bounds every one of them.  The
bf16 rounding is 2^-8 at most per element, 1.7e-3 in a norm, and most rows hold
no such code: 6e-3 bounds the median.  A row left out or written twice is off
by about 1.
"""
import pytest
import torch

import ref64 as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


def _at(ctx, p, n, f):
    off = p.value - ctx.ctx.data_ptr()
    return ctx.ctx[off:off + 2 * n * f].view(torch.bfloat16).view(n, f).double()


def _hold(got, want, what):
    for dim, name in ((1, "row"), (0, "column")):
        off = (got.double() - want).norm(dim=dim) / want.norm(dim=dim).clamp_min(1e-300)
        assert float(off.max()) <= 0.125, f"{what}: {name} {int(off.argmax())} off by {float(off.max()):.3g}"
        assert float(off.median()) <= 6e-3, f"{what}: {name}s off by {float(off.median()):.3g}"


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("recipe,N,K,F", [
    ("block", 129, 144, 128), ("block", 1000, 528, 384), ("block", 4113, 272, 512), ("block", 2049, 1040, 1152),
    ("tensorwise", 129, 144, 144), ("tensorwise", 1000, 528, 400), ("tensorwise", 4113, 272, 528),
    ("tensorwise", 2049, 1040, 1136)])
def test_every_row_and_column(fp, recipe, N, K, F, act):
    g = torch.Generator().manual_seed(N + K + F)
    x = torch.randn((N, K), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((2 * F, K), generator=g) * 2 / K ** 0.5).to(torch.bfloat16).cuda()
    dh = (torch.randn((N, F), generator=g) * 1e-2).to(torch.bfloat16).cuda()
    cache = fp.WeightCache()
    h = cache.register(w, recipe)
    cache.begin_cycle()
    cache.get(h)
    y, ctx = fp.fp8_gated_fwd(x, cache, h, recipe, act=act)
    dx, dw = fp.fp8_gated_bwd(dh, ctx, cache, h, recipe)
    xd = x.double()
    xq, wq = ref.operand(xd, recipe, "act"), ref.operand(w.double(), recipe, "weight")
    p = fp.fp8_gated_ctx_layout(recipe, ctx)
    G, Up, dhd = _at(ctx, p[3], N, F), _at(ctx, p[4], N, F), dh.double()
    a, d = ref.act(G, act)
    _hold(y, ref.act((xq @ wq.t())[:, :F], act)[0] * (xq @ wq.t())[:, F:], "H")
    dgu = torch.cat([dhd * Up * d, dhd * a], 1)
    if recipe == "block":
        row, col = ref.block_values(dgu, "e5m2"), ref.block_values(dgu.t().contiguous(), "e5m2")
        xcol = ref.block_values(xd.t().contiguous(), "e4m3")
    else:
        row = ref.tensor_values(dgu, "e5m2")
        col, xcol = row.t(), xq.t()
    _hold(dx, row @ wq, "dX")
    _hold(dw, col @ xcol.t(), "dW")
    assert fp.fp8_get_device_status() == 0
