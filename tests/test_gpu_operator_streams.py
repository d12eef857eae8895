"""Calls of the norm and the gated feed-forward on a stream other than the
current one: their own tensors are not memory that the current stream still
writes, or writes again while the call runs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


def _busy_blocks(sizes):
    """Blocks of these sizes that are free for the current stream's next tensors
    while writes to them are still queued there, behind a wait of some 20 ms."""
    torch.cuda._sleep(40_000_000)
    for n in sizes:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x55)


@pytest.mark.parametrize("recipe", ["block", "tensorwise"])
def test_own_tensors_are_no_memory_in_use(fp, recipe):
    n, d, F = 300, 512, 640
    g = torch.Generator().manual_seed(4)
    x, res = (torch.randn((n, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    dy = (torch.randn((n, F), generator=g) * 1e-2).to(torch.bfloat16).cuda()
    w = (torch.randn((2 * F, d), generator=g) * 0.05).to(torch.bfloat16).cuda()
    wn = torch.ones(d, device="cuda")
    cache = fp.WeightCache()
    h = cache.register(w, recipe)
    cache.begin_cycle()
    cache.get(h)

    def calls(stream):
        sizes = [0]
        if stream is not None:  # everything that the calls make, twice over
            sizes = [2 * n * d, n * d, 2 * n * F, 2 * 2 * F * d, 4 * n, 4 * n * 4, 4 * d * 3, 304 * d] * 2
            sizes += [t.numel() for t in (fp.gated_context(recipe, n, d, F, "cuda").ctx,
                                          fp.gated_workspace(recipe, n, d, F, "cuda"),
                                          fp.gated_workspace(recipe, n, d, F, "cuda", train=False),
                                          fp.rmsnorm_workspace(n, d, "cuda"))]
            torch.cuda.synchronize()
            _busy_blocks(sizes)
        o = fp.fp8_rmsnorm_fwd(x, wn, residual=res, bf16=True, stream=stream)
        y, ctx = fp.fp8_gated_fwd(o["y"], cache, h, recipe, stream=stream)
        y1, _ = fp.fp8_gated_fwd(o["y"], cache, h, recipe, train=False, stream=stream)
        dx, dw = fp.fp8_gated_bwd(dy, ctx, cache, h, recipe, stream=stream)
        dxn, dwn = fp.fp8_rmsnorm_bwd(dx, o["r"], o["rstd"], wn, stream=stream)
        return [o[k] for k in ("r", "rstd", "y", "row", "row_scale", "col", "col_scale")] + [y, y1, dx, dw, dxn, dwn]

    want = calls(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = calls(s)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    assert fp.fp8_get_device_status() == 0
