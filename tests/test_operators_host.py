"""What the Python calls of the norm, the gated feed-forward and clipping check
and allocate, on the host: nothing reaches a GPU (hostcalls.py)."""
import pytest
import torch

from hostcalls import Host, bf16


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


@pytest.fixture
def host(fp, monkeypatch):
    return Host(fp, monkeypatch)


def _weight(fp, recipe, F=256, K=256):
    cache = fp.WeightCache()
    h = cache.register(bf16(2 * F, K), recipe)
    return cache, h


# ---------------------------------------------------------------- contexts
@pytest.mark.parametrize("made,used", [("tensorwise", "block"), ("block", "tensorwise"), ("delayed", "block")])
def test_context_of_another_recipe(fp, host, made, used):
    """The layouts differ: a block context is larger and holds G and U elsewhere."""
    cache, h = _weight(fp, used)
    ctx = fp.gated_context(made, 40, 256, 256, "cuda")
    with pytest.raises(ValueError):
        fp.fp8_gated_fwd(bf16(40, 256), cache, h, used, ctx=ctx)
    with pytest.raises(ValueError):
        fp.fp8_gated_bwd(bf16(40, 256), ctx, cache, h, used)
    with pytest.raises(ValueError):
        fp.fp8_gated_ctx_layout(used, ctx)
    assert not host.calls


def test_context_without_a_recipe_is_held_to_its_size(fp, host):
    cache, h = _weight(fp, "block")
    need = fp.gated_context("block", 40, 256, 256, "cuda").ctx.numel()
    short = fp.GatedContext(torch.empty(need - 1, dtype=torch.uint8, device="cuda"), 40, 256, 256)
    with pytest.raises(ValueError):
        fp.fp8_gated_fwd(bf16(40, 256), cache, h, "block", ctx=short)
    with pytest.raises(ValueError):
        fp.fp8_gated_bwd(bf16(40, 256), short, cache, h, "block")
    assert not host.calls
    own = fp.GatedContext(torch.empty(need, dtype=torch.uint8, device="cuda"), 40, 256, 256)
    fp.fp8_gated_fwd(bf16(40, 256), cache, h, "block", ctx=own)
    fp.fp8_gated_bwd(bf16(40, 256), own, cache, h, "block")
    assert len(host.calls) == 2


def test_context_on_the_host(fp, host):
    cache, h = _weight(fp, "block")
    ctx = fp.gated_context("block", 40, 256, 256, "cuda")
    ctx.ctx = torch.zeros(ctx.ctx.numel(), dtype=torch.uint8)
    with pytest.raises(ValueError):
        fp.fp8_gated_fwd(bf16(40, 256), cache, h, "block", ctx=ctx)
    assert not host.calls


def test_delayed_and_tensorwise_contexts_are_alike(fp, host):
    cache, h = _weight(fp, "delayed")
    ctx = fp.gated_context("tensorwise", 40, 256, 256, "cuda")
    fp.fp8_gated_fwd(bf16(40, 256), cache, h, "delayed", ctx=ctx)
    fp.fp8_gated_bwd(bf16(40, 256), ctx, cache, h, "delayed")
    assert len(host.calls) == 2


def test_backward_with_a_weight_of_another_shape(fp, host):
    """2F agrees, K does not: dX and the transposed input have the weight's K."""
    cache, h = _weight(fp, "tensorwise", K=256)
    wide = cache.register(bf16(512, 512), "tensorwise")
    ctx = fp.gated_context("tensorwise", 40, 256, 256, "cuda")
    with pytest.raises(ValueError):
        fp.fp8_gated_bwd(bf16(40, 256), ctx, cache, wide, "tensorwise")
    with pytest.raises(ValueError):
        fp.fp8_gated_bwd(bf16(40, 256), ctx, cache, wide + 1, "tensorwise")
    assert not host.calls
    fp.fp8_gated_bwd(bf16(40, 256), ctx, cache, h, "tensorwise")
    assert len(host.calls) == 1
