"""What a gated forward pass leaves in its context: the transposed FP8 input with
both of its scale arrays, for few tokens and for many."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


@pytest.mark.parametrize("recipe", ["block", "tensorwise"])
@pytest.mark.parametrize("N,K", [(16, 16), (16, 4096), (48, 528), (64, 2048), (80, 528), (256, 1040)])
def test_transposed_input_and_scales(fp, recipe, N, K):
    F = 128
    g = torch.Generator().manual_seed(N + K)
    x = torch.randn((N, K), generator=g).to(torch.bfloat16).cuda()
    x[:, K // 2] = 0
    cache = fp.WeightCache()
    h = cache.register(torch.ones((2 * F, K), dtype=torch.bfloat16, device="cuda"), recipe)
    cache.begin_cycle()
    cache.get(h)
    ctx = fp.gated_context(recipe, N, K, F, "cuda")
    ctx.ctx.fill_(0xFF)
    fp.fp8_gated_fwd(x, cache, h, recipe, ctx=ctx)
    q = fp.fp8_quantize(x, recipe, "act")
    p = fp.fp8_gated_ctx_layout(recipe, ctx)

    def at(ptr, like):
        off = ptr.value - ctx.ctx.data_ptr()
        n = like.numel() * like.element_size()
        return ctx.ctx[off:off + n].view(like.dtype).view(like.shape)

    for ptr, key in zip(p, ("col", "col_scale", "col_scale_inv")):
        assert torch.equal(at(ptr, q[key]), q[key]), key
