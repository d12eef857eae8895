"""Gated feed-forward, forward and backward, against a plain 64-bit statement.

Tolerances, with u = 2^-24 and v = 2^-8 (bf16, 8 significand bits):
  * the quantized operands equal the definition bit for bit, so G and U differ
    by fp32 summation alone: within K u of the sum of magnitudes (e_G, e_U);
  * H = act(G) U: |act'| <= 1.13, so 1.2 e_G |U| + |act(G)| e_U, 2e-5 of |H|
    for the activation's approximations, and one bf16 rounding;
  * kept projections: e_G (e_U) and one bf16 rounding;
  * gradients: dG and dU are formed from the kept projections in fp32, a few u
    off, so an E5M2 code differs only for values within that of a tie: about
    2e-6 of the elements, a quarter of such an element each.  Ten such codes
    among the 256 or more terms of each output, over all rows, and the bf16
    rounding of the outputs (1.7e-3 in this norm) stay below 5e-3.
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


def _case(fp, N, K, F, recipe, seed=0):
    g = torch.Generator().manual_seed(seed + N + K + F)
    x = torch.randn((N, K), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((2 * F, K), generator=g) * 2 / K ** 0.5).to(torch.bfloat16).cuda()
    dh = (torch.randn((N, F), generator=g) * 1e-2).to(torch.bfloat16).cuda()
    cache = fp.WeightCache()
    h = cache.register(w, recipe)
    cache.begin_cycle()
    cache.get(h)
    return x, w, dh, cache, h


def _tensor_at(ptr, shape, base):
    """The bf16 tensor that a context holds at a device pointer."""
    off = ptr.value - base.data_ptr()
    n = shape[0] * shape[1] * 2
    return base[off:off + n].view(torch.bfloat16).view(shape)


def _rel(a, b):
    n = float(b.norm())
    return float((a.double() - b).norm()) / n if n else float(a.double().norm())


def _check(fp, N, K, F, recipe, act, seed=0):
    x, w, dh, cache, h = _case(fp, N, K, F, recipe, seed)
    ref_recipe = "block" if recipe == "block" else "tensorwise"
    xd, wd = x.double(), w.double()
    xq, wq = ref.operand(xd, ref_recipe, "act"), ref.operand(wd, ref_recipe, "weight")
    gu, mag = xq @ wq.t(), K * U * (xq.abs() @ wq.abs().t())
    G, Up, eG, eU = gu[:, :F], gu[:, F:], mag[:, :F], mag[:, F:]
    a, _ = ref.act(G, act)
    H = a * Up
    tol = 1.2 * eG * Up.abs() + a.abs() * eU + eG * eU + (2e-5 + ref.EPS8) * H.abs() + 1e-37
    y, none = fp.fp8_gated_fwd(x, cache, h, recipe, act=act, train=False)
    assert none is None
    assert torch.all((y.double() - H).abs() <= tol), "inference output"
    y2, ctx = fp.fp8_gated_fwd(x, cache, h, recipe, act=act)
    assert torch.all((y2.double() - H).abs() <= tol), "training output"
    p = fp.fp8_gated_ctx_layout(recipe, ctx)
    kept = torch.cat([_tensor_at(p[3], (N, F), ctx.ctx), _tensor_at(p[4], (N, F), ctx.ctx)], 1)
    assert torch.all((kept.double() - gu).abs() <= mag * (1 + ref.EPS8) + ref.EPS8 * gu.abs() + 1e-38), "kept"
    k = kept.double()
    ka, kd = ref.act(k[:, :F], act)
    dhd = dh.double()
    dgu = torch.cat([dhd * k[:, F:] * kd, dhd * ka], 1)
    dx, dw = fp.fp8_gated_bwd(dh, ctx, cache, h, recipe)
    if ref_recipe == "block":
        row = ref.block_values(dgu, "e5m2")
        col = ref.block_values(dgu.t().contiguous(), "e5m2")
        xcol = ref.block_values(xd.t().contiguous(), "e4m3")
    else:
        row = ref.tensor_values(dgu, "e5m2")
        col, xcol = row.t(), xq.t()
    assert _rel(dx, row @ wq) <= 5e-3, "dx"
    assert _rel(dw, col @ xcol.t()) <= 5e-3, "dw"
    none, dw2 = fp.fp8_gated_bwd(dh, ctx, cache, h, recipe, need_dx=False)
    assert none is None and torch.equal(dw, dw2)
    assert fp.fp8_get_device_status() == 0


@pytest.mark.parametrize("N,K,F", [(1, 16, 128), (1, 512, 256), (2, 144, 384), (7, 4096, 256), (16, 128, 128),
                                   (37, 272, 512), (64, 1024, 640), (65, 1040, 384), (128, 256, 256),
                                   (129, 384, 128), (300, 512, 1024), (1000, 2064, 384)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_block(fp, N, K, F, act):
    _check(fp, N, K, F, "block", act)


@pytest.mark.parametrize("N,K,F", [(1, 16, 16), (1, 512, 2048), (3, 144, 48), (16, 64, 80), (37, 512, 400),
                                   (64, 4096, 1040), (65, 528, 112), (127, 256, 272), (257, 384, 144),
                                   (1000, 1040, 560), (2100, 4096, 272)])
@pytest.mark.parametrize("recipe,act", [("tensorwise", "silu"), ("tensorwise", "gelu"), ("delayed", "silu")])
def test_tensorwise(fp, N, K, F, recipe, act):
    if recipe == "delayed":
        # the first quantization of a weight with an empty history has scale 1,
        # which is not the definition above: use one with a history
        x, w, dh, cache, h = _case(fp, N, K, F, recipe)
        cache.begin_cycle()
        cache.get(h)
        y, ctx = fp.fp8_gated_fwd(x, cache, h, recipe, act=act)
        dx, dw = fp.fp8_gated_bwd(dh, ctx, cache, h, recipe)
        _, _, _, c2, h2 = _case(fp, N, K, F, "tensorwise")
        y2, ctx2 = fp.fp8_gated_fwd(x, c2, h2, "tensorwise", act=act)
        dx2, dw2 = fp.fp8_gated_bwd(dh, ctx2, c2, h2, "tensorwise")
        assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
        return
    _check(fp, N, K, F, recipe, act)


def test_few_tokens_over_a_very_deep_product(fp):
    """More K blocks than the few-token kernel takes in one CTA."""
    _check(fp, 3, 66048, 128, "block", "silu")


@pytest.mark.parametrize("recipe", ["tensorwise", "block"])
def test_several_waves(fp, recipe):
    """More output tiles than the GPU has SMs, so every ring and accumulator
    buffer is used many times over."""
    _check(fp, 4500, 1152, 1536, recipe, "silu")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_derivative_formula_against_differences(act):
    g = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    h = 1e-5
    num = (ref.act(g + h, act)[0] - ref.act(g - h, act)[0]) / (2 * h)
    assert float((num - ref.act(g, act)[1]).abs().max()) < 1e-9


def test_gradients_follow_differences(fp):
    """Directional derivatives of sum(dH * H) without any quantization, in 64
    bits, against the kernels' gradients.  E4M3 operands and E5M2 gradients
    carry up to 2^-4 and 2^-3 of relative error per element, independent of
    each other, so 5% of the terms' root sum of squares bounds the sum."""
    N, K, F = 200, 256, 384
    x, w, dh, cache, h = _case(fp, N, K, F, "block", 3)
    y, ctx = fp.fp8_gated_fwd(x, cache, h, "block")
    dx, dw = fp.fp8_gated_bwd(dh, ctx, cache, h, "block")
    xd, wd, dhd = x.double(), w.double(), dh.double()

    def loss(x, w):
        gu = x @ w.t()
        return (dhd * ref.act(gu[:, :F], "silu")[0] * gu[:, F:]).sum()

    xr, wr = xd.clone().requires_grad_(), wd.clone().requires_grad_()
    loss(xr, wr).backward()
    for got, exact, at, other in ((dx, xr.grad, xd, lambda t: loss(t, wd)), (dw, wr.grad, wd, lambda t: loss(xd, t))):
        v = exact / exact.norm()
        e = 1e-4
        d = float((other(at + e * v) - other(at - e * v)) / (2 * e))
        assert abs(d - float(exact.norm())) < 1e-5 * d  # the differences agree with the exact gradient
        assert abs(float((got.double() * v).sum()) - d) < 0.05 * d
        assert _rel(got, exact) < 0.15


def test_extreme_projections(fp):
    """Large negative and positive gates: silu and its derivative stay finite
    and reach their limits; zero inputs give zeros."""
    F, K = 128, 128
    w = torch.zeros((2 * F, K), dtype=torch.bfloat16, device="cuda")
    w[:F, 0] = torch.linspace(-300, 300, F).to(torch.bfloat16)
    w[F:, 1] = 1.0
    x = torch.zeros((20, K), dtype=torch.bfloat16, device="cuda")
    x[:10, 0] = 1.0
    x[:10, 1] = 1.0
    cache = fp.WeightCache()
    h = cache.register(w, "tensorwise")
    cache.begin_cycle()
    cache.get(h)
    for act in ("silu", "gelu"):
        y, ctx = fp.fp8_gated_fwd(x, cache, h, "tensorwise", act=act)
        assert bool(torch.isfinite(y).all()) and int(y[10:].count_nonzero()) == 0
        wq = ref.tensor_values(w.double(), "e4m3")
        want = ref.act(wq[:F, 0], act)[0] * wq[F:, 1]
        assert torch.all((y[0].double() - want).abs() <= (ref.EPS8 + 2e-5) * want.abs() + 1e-30)
        dx, dw = fp.fp8_gated_bwd(torch.ones_like(y), ctx, cache, h, "tensorwise")
        assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())


def test_quantized_input_from_the_norm(fp):
    """The norm's FP8 output feeds both directions without a bf16 copy: equal
    to quantized operands given by hand."""
    N, K, F = 130, 256, 384
    x, w, dh, cache, h = _case(fp, N, K, F, "block", 5)
    nw = torch.ones(K, device="cuda")
    q = fp.fp8_rmsnorm_fwd(x, nw)
    ctx = fp.gated_context("block", N, K, F, "cuda")
    p = fp.fp8_gated_ctx_layout("block", ctx)
    base = ctx.ctx
    for ptr, src in ((p[0], q["col"]), (p[1], q["col_scale"]), (p[2], q["col_scale_inv"])):
        flat = src.contiguous().view(torch.uint8).view(-1)
        off = ptr.value - base.data_ptr()
        base[off:off + flat.numel()] = flat
    y, _ = fp.fp8_gated_fwd_quantized(q["row"], q["row_scale_inv"], cache, h, "block", ctx=ctx)
    xq = ref.decode(q["row"], "e4m3") * q["row_scale_inv"].double().repeat_interleave(128, 1)[:, :K]
    wq = ref.operand(w.double(), "block", "weight")
    gu = xq @ wq.t()
    assert _rel(y, ref.act(gu[:, :F], "silu")[0] * gu[:, F:]) <= 2.5e-3
    y2, none = fp.fp8_gated_fwd_quantized(q["row"], q["row_scale_inv"], cache, h, "block")
    assert none is None and torch.equal(y, y2)
    dx, dw = fp.fp8_gated_bwd(dh, ctx, cache, h, "block")
    k = torch.cat([_tensor_at(p[3], (N, F), base), _tensor_at(p[4], (N, F), base)], 1).double()
    a, d = ref.act(k[:, :F], "silu")
    dgu = torch.cat([dh.double() * k[:, F:] * d, dh.double() * a], 1)
    xcol = ref.decode(q["col"][:, :N].contiguous(), "e4m3") * q["col_scale_inv"].double().repeat_interleave(128, 1)[:, :N]
    assert _rel(dw, ref.block_values(dgu.t().contiguous(), "e5m2") @ xcol.t()) <= 5e-3


def test_no_tokens_and_side_stream(fp):
    x, w, dh, cache, h = _case(fp, 96, 256, 256, "block", 7)
    y, ctx = fp.fp8_gated_fwd(x[:0], cache, h, "block")
    assert y.shape == (0, 256)
    dx, dw = fp.fp8_gated_bwd(dh[:0], ctx, cache, h, "block")
    assert dx.shape == (0, 256) and int(dw.count_nonzero()) == 0
    want, ctx = fp.fp8_gated_fwd(x, cache, h, "block")
    wdx, wdw = fp.fp8_gated_bwd(dh, ctx, cache, h, "block")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, ctx = fp.fp8_gated_fwd(x, cache, h, "block")
        gdx, gdw = fp.fp8_gated_bwd(dh, ctx, cache, h, "block")
    s.synchronize()
    assert torch.equal(want, got) and torch.equal(wdx, gdx) and torch.equal(wdw, gdw)


def test_refusals(fp):
    x, w, dh, cache, h = _case(fp, 32, 256, 256, "block", 8)
    with pytest.raises(ValueError):
        fp.fp8_gated_fwd(x.float(), cache, h, "block")
    with pytest.raises(KeyError):
        fp.fp8_gated_fwd(x, cache, h, "block", act="relu")
    with pytest.raises(fp.FP8Error):
        fp.fp8_gated_fwd(x, cache, h, "tensorwise")       # not the registered recipe
    with pytest.raises(fp.FP8Error):
        fp.fp8_gated_fwd(x[:, :128].contiguous(), cache, h, "block")
    with pytest.raises(ValueError):
        fp.fp8_gated_fwd(x, cache, h + 1, "block")
    with pytest.raises(ValueError):
        fp.fp8_gated_fwd(x, cache, h, "block", y=torch.empty((32, 128), dtype=torch.bfloat16, device="cuda"))
    _, ctx = fp.fp8_gated_fwd(x, cache, h, "block")
    with pytest.raises(ValueError):
        fp.fp8_gated_bwd(dh[:16], ctx, cache, h, "block")
    with pytest.raises(fp.FP8Error):
        fp.fp8_gated_bwd(dh, ctx, cache, h, "block", ws=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    cache.begin_cycle()
    with pytest.raises(fp.FP8Error):                       # stale weight
        fp.fp8_gated_fwd(x, cache, h, "block")
    odd = cache.register(torch.zeros((320, 256), dtype=torch.bfloat16, device="cuda"), "block")
    cache.get(odd)
    with pytest.raises(fp.FP8Error):                       # F = 160: tiles would straddle Wg and Wu
        fp.fp8_gated_fwd(x, cache, odd, "block")


@pytest.mark.parametrize("recipe", ["tensorwise", "block"])
@pytest.mark.parametrize("N,K", [(16, 16), (16, 528), (32, 1040), (48, 2048), (64, 4096)])
def test_few_token_quantizer_equals_the_quantizer(fp, recipe, N, K):
    """The transposed FP8 input kept for the backward pass is that of
    fp8_quantize bit for bit, special values included."""
    F = 128
    x, w, dh, cache, h = _case(fp, N, K, F, recipe, 9)
    x[0, 0] = float("nan")
    x[N - 1, K - 1] = -float("inf") if recipe == "block" else 0.0
    x[3, :] = 0
    x[:, 5] = 0
    y, ctx = fp.fp8_gated_fwd(x, cache, h, recipe)
    q = fp.fp8_quantize(x, recipe, "act")
    p = fp.fp8_gated_ctx_layout(recipe, ctx)
    off = p[0].value - ctx.ctx.data_ptr()
    assert torch.equal(ctx.ctx[off:off + N * K].view(K, N), q["col"])
    off = p[2].value - ctx.ctx.data_ptr()
    si = q["col_scale_inv"]
    assert torch.equal(ctx.ctx[off:off + 4 * si.numel()].view(torch.float32).view(si.shape), si)


@pytest.mark.parametrize("N,K,F", [(1, 16, 16), (65, 128, 272), (5000, 128, 272), (555, 272, 128), (2003, 352, 176),
                                   (2217, 800, 2624), (10556, 272, 2960), (8246, 816, 2736), (23795, 288, 2560)])
def test_weight_gradient_from_the_row_layout(fp, N, K, F):
    """Tensor scaling keeps dGU in rows only: the product that reads them
    M-major equals, bit for bit, the GEMM on a transposed copy.  The sizes take
    every tile shape of the GEMM, with and without a split of the tokens."""
    x, w, dh, cache, h = _case(fp, N, K, F, "tensorwise", 11)
    y, ctx = fp.fp8_gated_fwd(x, cache, h, "tensorwise")
    ws = fp.gated_workspace("tensorwise", N, K, F, "cuda")
    ws.fill_(0xFF)
    dx, dw = fp.fp8_gated_bwd(dh, ctx, cache, h, "tensorwise", ws=ws)
    Np = (N + 15) // 16 * 16
    # the workspace begins with the rows, their scale_inv follows
    rows = N * 2 * F
    a = torch.zeros((2 * F, Np), dtype=torch.uint8, device="cuda")
    a[:, :N] = ws[:rows].view(N, 2 * F).t()
    sa = ws[-(-rows // 256) * 256:][:4].view(torch.float32)
    p = fp.fp8_gated_ctx_layout("tensorwise", ctx)
    off, sb = p[0].value - ctx.ctx.data_ptr(), p[2].value - ctx.ctx.data_ptr()
    xt = ctx.ctx[off:off + K * Np].view(K, Np)
    want = fp.fp8_gemm(a, "e5m2", sa, xt, "e4m3", ctx.ctx[sb:sb + 4].view(torch.float32), "tensor")
    assert torch.equal(dw, want)
    assert fp.fp8_get_device_status() == 0


@pytest.mark.parametrize("recipe", ["tensorwise", "block"])
@pytest.mark.parametrize("N,K,F", [(1, 16, 128), (1, 4096, 14336), (2, 4096, 1024), (7, 144, 256), (8, 528, 256),
                                   (9, 2064, 512), (16, 4096, 2048), (17, 1040, 128), (33, 512, 2048), (37, 512, 2048),
                                   (40, 400, 640), (57, 1552, 128), (64, 128, 256), (64, 2032, 512)])
def test_tokens_quantized_in_the_kernel(fp, recipe, N, K, F):
    """Without a backward pass few tokens go into the kernel as bf16: the same
    bits as through the quantizer, special values included."""
    x, w, dh, cache, h = _case(fp, N, K, F, recipe, 12)
    x[N // 2, K // 2] = 0.0
    x[N - 1, :] = 0.0
    if N > 2:
        x[1, 3] = float("nan")
    y, ctx = fp.fp8_gated_fwd(x, cache, h, recipe)
    y2, _ = fp.fp8_gated_fwd(x, cache, h, recipe, train=False)
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    if N > 3 and recipe == "block":
        x[2, K - 1] = float("inf")
        y, ctx = fp.fp8_gated_fwd(x, cache, h, recipe)
        y2, _ = fp.fp8_gated_fwd(x, cache, h, recipe, train=False)
        assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    assert fp.fp8_get_device_status() == 0
