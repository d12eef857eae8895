"""What the Python calls of the norm, the gated feed-forward and clipping check
and allocate, on the host: nothing reaches a GPU (hostcalls.py)."""
import pytest
import torch

from hostcalls import FakeStream, Host, bf16, dev, f32


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


# ---------------------------------------------------------------- quantized input
@pytest.mark.parametrize("bad", [
    dict(shape=(40, 1)), dict(shape=(39, 2)), dict(shape=(2, 40)), dict(shape=(79,)), dict(shape=(81,)),
    dict(dtype=torch.float64), dict(dtype=torch.bfloat16), dict(strided=True), dict(on_host=True)])
def test_scales_of_a_quantized_input(fp, host, bad):
    """The block kernel reads one float per token and 128 columns."""
    cache, h = _weight(fp, "block")
    row = dev(torch.zeros((40, 256), dtype=torch.uint8))
    s = torch.zeros(bad.get("shape", (40, 2)), dtype=bad.get("dtype", torch.float32))
    if bad.get("strided"):
        s = torch.zeros((40, 4))[:, ::2]
    with pytest.raises(ValueError):
        fp.fp8_gated_fwd_quantized(row, s if bad.get("on_host") else dev(s), cache, h, "block")
    assert not host.calls


@pytest.mark.parametrize("recipe,shape", [("block", (40, 2)), ("block", (80,)), ("tensorwise", (1,)),
                                          ("tensorwise", (1, 1)), ("tensorwise", ()), ("delayed", (1,))])
def test_scales_that_fit(fp, host, recipe, shape):
    cache, h = _weight(fp, recipe)
    fp.fp8_gated_fwd_quantized(dev(torch.zeros((40, 256), dtype=torch.uint8)), f32(*shape), cache, h, recipe)
    assert len(host.calls) == 1


def test_one_scale_for_the_tensorwise_recipe(fp, host):
    cache, h = _weight(fp, "tensorwise")
    with pytest.raises(ValueError):
        fp.fp8_gated_fwd_quantized(dev(torch.zeros((40, 256), dtype=torch.uint8)), f32(0), cache, h, "tensorwise")
    assert not host.calls


# ---------------------------------------------------------------- streams
def test_tensors_of_a_call_come_from_its_stream(fp, host):
    """What a call on another stream allocates (outputs, context, workspace) has
    to come from that stream's pool: a block just freed on the current stream may
    still be written by work queued there, and one freed right after the call
    may be handed to the current stream while the call's kernels use it."""
    s = FakeStream(77)
    cache, h = _weight(fp, "block")
    x, w, dh = bf16(40, 256), f32(256), bf16(40, 256)

    def only(stream, count):
        made, host.made[:] = list(host.made), []
        assert len(made) == count and all(at == stream for _, at in made)

    host.made.clear()
    for stream, at in ((s, 77), (None, 0)):
        o = fp.fp8_rmsnorm_fwd(x, w, residual=x, bf16=True, stream=stream)
        only(at, 10)
        fp.fp8_rmsnorm_bwd(dh, x, o["rstd"], w, stream=stream)
        only(at, 3)
        fp.fp8_gated_fwd(x, cache, h, "block", train=False, stream=stream)
        only(at, 2)
        _, ctx = fp.fp8_gated_fwd(x, cache, h, "block", stream=stream)
        only(at, 3)
        fp.fp8_gated_bwd(dh, ctx, cache, h, "block", stream=stream)
        only(at, 3)
        fp.fp8_gated_fwd_quantized(o["row"], o["row_scale_inv"], cache, h, "block", stream=stream)
        only(at, 1)
    assert host.on == []


def test_buffers_given_are_not_made_again(fp, host):
    cache, h = _weight(fp, "block")
    x, dh = bf16(40, 256), bf16(40, 256)
    y, ctx = bf16(40, 256), fp.gated_context("block", 40, 256, 256, "cuda")
    ws = fp.gated_workspace("block", 40, 256, 256, "cuda")
    dx, dw = bf16(40, 256), bf16(512, 256)
    host.made.clear()
    s = FakeStream(77)
    assert fp.fp8_gated_fwd(x, cache, h, "block", ws=ws, y=y, ctx=ctx, stream=s) == (y, ctx)
    fp.fp8_gated_bwd(dh, ctx, cache, h, "block", ws=ws, dx=dx, dw=dw, stream=s)
    assert host.made == [] and [a[-1] for _, a in host.calls] == [77, 77]


# ---------------------------------------------------------------- clipping
def test_plan_of_a_clipping_run_on_other_streams(fp, host):
    """The plan's own memory is recorded on every stream that a call uses: a plan
    dropped while a call is pending must not give its pointer table away."""
    c = fp.GradClip([f32(100)])
    table, ws = c._table, c._ws
    c.clip(1.0)
    assert not table.recorded and not ws.recorded  # made on this stream
    c.clip(1.0, stream=FakeStream(5))
    c.norm(stream=FakeStream(6))
    host.current = 9                                # the caller's current stream has changed
    c.clip(1.0)
    c.clip(1.0, stream=FakeStream(5))
    assert table.recorded == ws.recorded == [5, 6, 9]
    assert [a[-1] for _, a in host.calls] == [0, 5, 6, 9, 5]


def test_plan_memory_is_ready_for_every_stream(fp, host):
    """The table's upload returns when it is done, and all earlier work of its
    stream with it; the workspace made before it is then free of such work too."""
    host.made.clear()
    c = fp.GradClip([f32(100)])
    order = [t.data_ptr() for t, _ in host.made]
    assert order.index(c._ws.data_ptr()) < order.index(c._table.data_ptr())


# ---------------------------------------------------------------- norm buffers

@pytest.mark.parametrize("change", [
    lambda b, t: b.__setitem__("row", t), lambda b, t: b.update(row=t), lambda b, t: b.update({"row": t}),
    lambda b, t: b.__ior__({"row": t}), lambda b, t: (b.pop("row"), b.setdefault("row", t)),
    lambda b, t: (b.__delitem__("row"), b.setdefault("row", t)),
    lambda b, t: (lambda rest: (b.clear(), rest.update(row=t), [b.setdefault(k, v) for k, v in rest.items()]))(dict(b))])
def test_every_change_of_the_buffers_is_checked(fp, host, change):
    x, w = bf16(40, 256), f32(256)
    buf = fp.rmsnorm_buffers(40, 256, "cuda")
    fp.fp8_rmsnorm_fwd(x, w, residual=x, out=buf)
    assert len(host.calls) == 1 and buf.checked is not None
    change(buf, torch.empty((4, 128), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_fwd(x, w, residual=x, out=buf)
    assert len(host.calls) == 1


@pytest.mark.parametrize("gone", [lambda b: b.pop("col"), lambda b: b.__delitem__("col"), lambda b: b.clear(),
                                  lambda b: [b.popitem() for _ in range(3)]])
def test_buffers_taken_out(fp, host, gone):
    x, w = bf16(40, 256), f32(256)
    buf = fp.rmsnorm_buffers(40, 256, "cuda")
    fp.fp8_rmsnorm_fwd(x, w, residual=x, out=buf)
    gone(buf)
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_fwd(x, w, residual=x, out=buf)
    assert len(host.calls) == 1


def test_result_without_a_residual_holds_no_buffer_for_the_stream(fp, host):
    """There r is the caller's x: given back as `out` of a call with a residual it
    must not be written over."""
    x, w = bf16(40, 256), f32(256)
    o = fp.fp8_rmsnorm_fwd(x, w)
    assert o["r"] is x
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_fwd(bf16(40, 256), w, residual=bf16(40, 256), out=o)
    assert len(host.calls) == 1
    p = fp.fp8_rmsnorm_fwd(bf16(40, 256), w, out=o)  # without one nothing is written there
    q = fp.fp8_rmsnorm_fwd(bf16(40, 256), w, out=p)
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_fwd(bf16(40, 256), w, residual=bf16(40, 256), out=q)
    r = bf16(40, 256)
    o["r"] = r                                       # now it does
    assert fp.fp8_rmsnorm_fwd(x, w, residual=x, out=o)["r"] is r
    assert host.launches("fp8_rmsnorm_fwd")[-1][7] == r.data_ptr()
    p.update(r=r)
    assert fp.fp8_rmsnorm_fwd(x, w, residual=x, out=p)["r"] is r


def test_buffers_of_the_outputs_asked_for_are_enough(fp, host):
    x, w = bf16(40, 256), f32(256)
    o = fp.fp8_rmsnorm_fwd(x, w, rowwise=False, colwise=False, bf16=True, out=dict(rstd=f32(40), y=bf16(40, 256)))
    assert o["r"] is x and o["y"].shape == (40, 256)
    row = dict(rstd=f32(40), row=dev(torch.zeros((40, 256), dtype=torch.uint8)), row_scale=f32(40, 2),
               row_scale_inv=f32(40, 2), r=bf16(40, 256))
    fp.fp8_rmsnorm_fwd(x, w, residual=x, colwise=False, out=row)
    assert len(host.calls) == 2


def test_every_call_returns_a_norm_of_its_own(fp, host):
    """A caller that collects the norms of several steps reads them later."""
    c = fp.GradClip([f32(100)])
    host.made.clear()
    a, _ = c.clip(1.0)
    b = c.norm()
    d, _ = c.clip(1.0, stream=FakeStream(5))
    assert len({t.data_ptr() for t in (a, b, d)}) == 3
    assert [at for _, at in host.made] == [0, 5] and host.made[1][0].data_ptr() == d.data_ptr()
    assert all(t.shape == (1,) and t.dtype == torch.float32 for t in (a, b, d))
    assert [args[3] for args in host.launches("fp8_grad_clip_run")] == [a.data_ptr(), d.data_ptr()]
    assert [args[2] for args in host.launches("fp8_grad_norm")] == [b.data_ptr()]


# ---------------------------------------------------------------- devices and workspaces
def test_workspaces_on_the_host_are_refused(fp, host):
    cache, h = _weight(fp, "block")
    x, dh, w = bf16(40, 256), bf16(40, 256), f32(256)
    _, ctx = fp.fp8_gated_fwd(x, cache, h, "block")
    n = len(host.calls)
    ws = torch.zeros(1 << 24, dtype=torch.uint8)
    for call in (lambda: fp.fp8_gated_fwd(x, cache, h, "block", ws=ws),
                 lambda: fp.fp8_gated_bwd(dh, ctx, cache, h, "block", ws=ws),
                 lambda: fp.fp8_rmsnorm_bwd(x, x, f32(40), w, ws=ws)):
        with pytest.raises(ValueError):
            call()
        ws2 = dev(torch.zeros((1 << 12, 1 << 12), dtype=torch.uint8))[:, ::2]
        ws, ws2 = ws2, ws
        with pytest.raises(ValueError):
            call()
        ws = ws2
    assert len(host.calls) == n


def test_workspaces_count_bytes(fp, host):
    """A float32 workspace of as many bytes serves."""
    cache, h = _weight(fp, "block")
    x = bf16(40, 256)
    need = fp.gated_workspace("block", 40, 256, 256, "cuda", train=False).numel()
    fp.fp8_gated_fwd(x, cache, h, "block", train=False, ws=f32(need // 4))
    assert host.calls[-1][1][-2] == need


def test_tensors_of_another_device_are_refused(fp, host):
    cache, h = _weight(fp, "block")
    x, dh, w, rstd = bf16(40, 256), bf16(40, 256), f32(256), f32(40)
    _, ctx = fp.fp8_gated_fwd(x, cache, h, "block")
    n = len(host.calls)

    def away(t):
        return dev(t.clone(), 1)

    u8 = dev(torch.zeros((40, 256), dtype=torch.uint8))
    for call in (lambda: fp.fp8_rmsnorm_fwd(x, away(w)), lambda: fp.fp8_rmsnorm_fwd(x, w, residual=away(x)),
                 lambda: fp.fp8_rmsnorm_fwd(away(x), w, out=fp.rmsnorm_buffers(40, 256, "cuda", residual=False)),
                 lambda: fp.fp8_rmsnorm_bwd(x, away(x), rstd, w), lambda: fp.fp8_rmsnorm_bwd(x, x, away(rstd), w),
                 lambda: fp.fp8_rmsnorm_bwd(x, x, rstd, w, ws=away(u8)),
                 lambda: fp.fp8_gated_fwd(away(x), cache, h, "block", y=bf16(40, 256)),
                 lambda: fp.fp8_gated_fwd(x, cache, h, "block", ws=away(u8)),
                 lambda: fp.fp8_gated_fwd_quantized(u8, away(f32(40, 2)), cache, h, "block"),
                 lambda: fp.fp8_gated_bwd(away(dh), ctx, cache, h, "block", dx=bf16(40, 256), dw=bf16(512, 256)),
                 lambda: fp.fp8_gated_bwd(dh, ctx, cache, h, "block", dx=away(x)),
                 lambda: fp.GradClip([f32(8), away(f32(8))]), lambda: fp.GradClip([f32(8)], [away(f32(8))])):
        with pytest.raises(ValueError):
            call()
    assert len(host.calls) == n


def test_norms_share_one_allocation_of_their_stream(fp, host, monkeypatch):
    """Norms are handed out of blocks (an allocation per call took as long as the
    call), each block of one stream; a captured call makes its own in the graph's
    pool, which outlives it."""
    c = fp.GradClip([f32(100)])
    host.made.clear()
    first = [c.clip(1.0)[0] for _ in range(130)]
    assert len({t.data_ptr() for t in first}) == 130 and len(host.made) == 3
    host.current = 9
    c.norm()
    assert len(host.made) == 4 and host.made[-1][1] == 9
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: True, raising=False)
    a, b = c.norm(), c.norm()
    assert len(host.made) == 6 and a.data_ptr() == host.made[-2][0].data_ptr() != b.data_ptr()


def test_clipped_tensors_that_overlap_are_refused(fp, host):
    """The same memory scaled by two chunks at once: neither order nor factor
    would be certain.  Reading one tensor twice is fine."""
    g, o = f32(4096), f32(4096)
    a = dev(torch.zeros(8192))
    for grads, out in (([g, g], None), ([g, g[100:200]], None), ([g, f32(4096)], [o, o]), ([a[:4096]], [a[1:4097]]),
                       ([a[:4096], a[4096:]], [a[4096:], a[:4096]]), ([g, o], [f32(4096), g]),
                       ([a[:100], a[50:150]], [f32(100), a[50:150]])):
        with pytest.raises(ValueError):
            fp.GradClip(grads, out)
    fp.GradClip([g, g], [f32(4096), o])
    fp.GradClip([a[:4096], a[4096:], a[5:5]])
    fp.GradClip([a[:4096]], [a[4096:]])
    fp.GradClip([g, f32(0), f32(0)])


# ---------------------------------------------------------------- the linear's calls
def test_tensors_of_the_linear_calls_come_from_their_stream(fp, host):
    s = FakeStream(77)
    cache, h = _weight(fp, "block")
    x, dy = bf16(48, 256), bf16(48, 512)
    u8 = dev(torch.zeros((48, 256), dtype=torch.uint8))

    def only(at, count):
        made, host.made[:] = list(host.made), []
        assert len(made) == count and all(a == at for _, a in made)

    host.made.clear()
    for stream, at in ((s, 77), (None, 0)):
        for recipe, count in (("block", 7), ("tensorwise", 7)):
            fp.fp8_quantize(x, recipe, "act", stream=stream)
            only(at, count)
        fp.fp8_quantize_delayed(x, "act", f32(16), 0, stream=stream)
        only(at, 5)
        fp.fp8_gemm(u8, "e4m3", f32(1), u8, "e4m3", f32(1), "tensor", stream=stream)
        only(at, 2)
        _, ctx = fp.fp8_linear_fwd(x, cache, h, "block", stream=stream)
        only(at, 3)
        fp.fp8_linear_bwd(dy, ctx, cache, h, "block", stream=stream)
        only(at, 3)
        a = fp.fp8_gelu_fwd(x, stream=stream)
        only(at, 1)
        fp.fp8_gelu_bwd(a, x, stream=stream)
        only(at, 1)
