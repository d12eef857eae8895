"""Products with 4-bit weights against a plain statement in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative


@pytest.fixture(scope="module", autouse=True)
def fp():
    import fp8_mixed_precision_gb300 as fp
    fp.lib()
    return fp


def weight(fp, shape, group, zero, seed):
    """A random weight on the GPU and its values in 64 bits on the CPU."""
    g = torch.Generator().manual_seed(seed)
    K = shape[-1]
    nb = -(-K // group)
    codes = torch.randint(0, 256, (*shape[:-1], K // 2), generator=g, dtype=torch.uint8)
    scale = (torch.rand((*shape[:-1], nb), generator=g) * 0.02 + 0.001).bfloat16()
    z = torch.randint(0, 16, (*shape[:-1], nb), generator=g, dtype=torch.uint8) if zero else None
    at = torch.arange(K) // group
    q = torch.stack((codes % 16, codes // 16), -1).flatten(-2).double()
    v = (q - (8.0 if z is None else z.double()[..., at])) * scale.double()[..., at]
    return fp.W4Weight(codes.cuda(), scale.cuda(), None if z is None else z.cuda(), group), v


def product(x, v):
    """x W^T and the bound of its error: products exact in fp32 within a group,
    sums of K terms in an order of their own (the tensor core's sums are not
    rounded to nearest: two units each), one scale per group."""
    y, size = x @ v.transpose(-1, -2), x.abs() @ v.abs().transpose(-1, -2)
    return y, size * (2 * v.shape[-1] / 16 + 64) * U


def act64(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    phi = torch.special.erfc(-g / math.sqrt(2)) / 2
    return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def gated(x, v, act):
    """h in 64 bits and its bound before the rounding to bf16: |act'| <= 1.13, and
    the activation itself within 2^-20 of the gate's size."""
    F = v.shape[0] // 2
    gu, eb = product(x, v)
    g, u = gu[:, :F], gu[:, F:]
    a, _ = act64(g, act)
    ea = 1.13 * eb[:, :F] + g.abs() * 2.0 ** -20
    return a * u, ea * (u.abs() + eb[:, F:]) + a.abs() * eb[:, F:] + (a * u).abs() * 4 * U


SHAPES = [(16, 32), (32, 64), (48, 96), (64, 512), (272, 288), (512, 2048), (2048, 512), (80, 4128), (16, 14336), (4096, 4608), (32, 40960)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
def test_linear(fp, N, K, group, zero):
    w, v = weight(fp, (N, K), group, zero, N + K)
    for T in (1, 2, 7, 8, 9, 16, 17, 33, 70):
        g = torch.Generator().manual_seed(T)
        x = torch.randn((T, K), generator=g).bfloat16()
        out = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
        y = fp.fp8_w4_linear(x.cuda(), w, out=out[:T])
        want, bound = product(x.double(), v)
        off = (y.cpu().double() - want).abs()
        assert bool((off <= bound + want.abs() * UB + 1e-38).all()), (T, float((off - want.abs() * UB).max()))
        assert bool((out[T] == 7.0).all())


@pytest.mark.parametrize("F,K", [(16, 32), (48, 512), (2048, 512), (144, 4096), (512, 8224), (16, 36864)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated(fp, F, K, group, act):
    w, v = weight(fp, (2 * F, K), group, group == 64, F + K)
    for T in (1, 5, 12, 64):
        g = torch.Generator().manual_seed(T + 1)
        x = torch.randn((T, K), generator=g).bfloat16()
        h = fp.fp8_w4_gated(x.cuda(), w, act).cpu().double()
        want, bound = gated(x.double(), v, act)
        assert bool(((h - want).abs() <= (bound + want.abs() * UB) * 1.01 + 1e-38).all())


def test_exact_values(fp):
    """One-hot tokens read every weight: each value exactly as it is defined."""
    for group in (32, 64, 128):
        for zero in (False, True):
            w, v = weight(fp, (48, 320), group, zero, 7)
            x = torch.eye(320, dtype=torch.bfloat16)
            y = fp.fp8_w4_linear(x.cuda(), w).cpu()
            assert torch.equal(y, v.t().bfloat16())


def test_nonfinite_stays_in_its_row(fp):
    w, v = weight(fp, (64, 512), 64, False, 3)
    x = torch.randn((9, 512)).bfloat16()
    x[4, 300] = math.inf
    x[6, 5] = math.nan
    y = fp.fp8_w4_linear(x.cuda(), w).cpu()
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[keep], fp.fp8_w4_linear(x[keep].contiguous().cuda(), w).cpu())
    assert bool(y[6].isnan().all()) and not bool(y[4].isfinite().any())


@pytest.mark.parametrize("T,E,k,K,F,N", [(1, 1, 1, 32, 32, 16), (1, 8, 2, 512, 256, 512), (1, 3, 4, 96, 64, 48),
                                         (5, 4, 2, 512, 96, 512), (37, 32, 4, 256, 128, 256), (3, 64, 2, 128, 64, 128),
                                         (70, 2, 1, 544, 160, 64), (64, 5, 3, 512, 2048, 512), (700, 4, 3, 64, 32, 32),
                                         (1, 2, 2, 64, 36864, 32), (9, 2, 2, 36864, 32, 32), (40, 3, 2, 4096, 4096, 64)])
@pytest.mark.parametrize("group,zero,act", [(32, True, "silu"), (64, False, "gelu"), (128, True, "silu")])
@pytest.mark.parametrize("kind", ["random", "holes"])
def test_experts(fp, T, E, k, K, F, N, group, zero, act, kind):
    gu, vgu = weight(fp, (E, 2 * F, K), group, zero, T + E)
    dn, vdn = weight(fp, (E, N, F), group, zero, T + F)
    g = torch.Generator().manual_seed(T * k)
    x = torch.randn((T, K), generator=g).bfloat16()
    e = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    w = torch.rand((T, k), generator=g)
    if kind == "holes":
        e[torch.rand((T, k), generator=g) < 0.4] = -1
        e[T - 1] = E + 5
    out = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = fp.fp8_w4_experts(x.cuda(), w.cuda(), e.cuda(), gu, dn, act, out=out[:T])
    want, bound = torch.zeros((T, N), dtype=torch.float64), torch.zeros((T, N), dtype=torch.float64)
    for i in range(E):
        t, j = (e == i).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        h, eh = gated(x.double()[t], vgu[i], act)
        eh = eh * 1.01 + h.abs() * UB * 1.01  # the rounding of h to bf16
        z, ez = product(h, vdn[i])
        ez = ez * (1 + UB) + eh @ vdn[i].abs().t()
        ww = w.double()[t, j][:, None]
        want.index_add_(0, t, ww * z)
        bound.index_add_(0, t, ww * (ez + z.abs() * (k + 2) * U))
    off = (y.cpu().double() - want).abs()
    assert bool((off <= bound + want.abs() * UB + 1e-38).all()), float((off / (bound + want.abs() * UB + 1e-38)).max())
    assert bool((out[T] == 7.0).all())
    again = fp.fp8_w4_experts(x.cuda(), w.cuda(), e.cuda(), gu, dn, act)
    assert torch.equal(again, y)


def test_routing_failure_shows(fp):
    """The row of a token with NaN weights is NaN, others are untouched by it."""
    gu, _ = weight(fp, (2, 64, 64), 32, False, 1)
    dn, _ = weight(fp, (2, 32, 32), 32, False, 2)
    x = torch.randn((3, 64), device="cuda").bfloat16()
    e = torch.tensor([[0, 1], [-1, -1], [1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.5], [math.nan, math.nan], [1.0, 0.0]], device="cuda")
    y = fp.fp8_w4_experts(x, w, e, gu, dn)
    assert bool(y[1].isnan().all()) and bool(y[0].isfinite().all()) and bool(y[2].isfinite().all())
    one = fp.fp8_w4_experts(x[1:2], w[1:2], e[1:2], gu, dn)
    assert bool(one.isnan().all())
    none = fp.fp8_w4_experts(x[:1], torch.zeros((1, 2), device="cuda"), e[1:2], gu, dn)
    assert bool((none == 0).all())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("shape", [(16, 32), (48, 416), (3, 32, 512)])
def test_quantize(fp, group, zero, shape):
    g = torch.Generator().manual_seed(group)
    w = torch.randn(shape, generator=g).bfloat16()
    w.view(-1, shape[-1])[1] = 0
    w.view(-1, shape[-1])[2] = w.view(-1, shape[-1])[2].abs()
    q = fp.fp8_w4_quantize(w.cuda(), group, zero)
    K, nb = shape[-1], -(-shape[-1] // group)
    pad = torch.zeros((*shape[:-1], nb * group))
    pad[..., :K] = w.float()
    p = pad.view(*shape[:-1], nb, group)
    hi, lo = p.amax(-1).clamp(min=0), p.amin(-1).clamp(max=0)
    s = ((hi - lo) / 15 if zero else torch.maximum(hi, -lo) / 7).bfloat16().float()
    s = torch.where(s == 0, torch.ones_like(s), s)
    z = (-lo / s).round().clamp(0, 15) if zero else torch.full_like(s, 8.0)
    c = ((p / s[..., None]).round() + z[..., None]).clamp(0, 15).view(*shape[:-1], -1)[..., :K].to(torch.uint8)
    assert torch.equal(q.scale.cpu().float(), s)
    assert torch.equal(q.codes.cpu(), c[..., 0::2] | c[..., 1::2] << 4)
    assert (q.zero is None) == (not zero) and (not zero or torch.equal(q.zero.cpu().float(), z))


def test_streams_and_graph(fp):
    gu, _ = weight(fp, (8, 128, 256), 64, True, 1)
    dn, _ = weight(fp, (8, 256, 64), 64, True, 2)
    x = torch.randn((6, 256), device="cuda").bfloat16()
    logits = torch.randn((6, 8), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    w, e = fp.fp8_route_fwd(logits, 2, stream=s)
    y = fp.fp8_w4_experts(x, w, e, gu, dn, stream=s)
    s.synchronize()
    w2, e2 = fp.fp8_route_fwd(logits, 2)
    ws = fp.w4_experts_workspace(6, 2, gu, dn)
    out = fp.fp8_w4_experts(x, w2, e2, gu, dn, ws=ws)
    assert torch.equal(out, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp.fp8_route_fwd(logits, 2, out=(w2, e2))
        fp.fp8_w4_experts(x, w2, e2, gu, dn, ws=ws, out=out)
    for _ in range(3):
        logits.normal_()
        x.normal_()
        g.replay()
        ww, ee = fp.fp8_route_fwd(logits, 2)
        assert torch.equal(out, fp.fp8_w4_experts(x, ww, ee, gu, dn))


def test_weights_past_32_bits(fp):
    """Codes past 2^31 bytes of a stack, its last expert alone in use."""
    E, N, F = 40, 4096, 28672
    codes = torch.zeros((E, N, F // 2), dtype=torch.uint8, device="cuda")
    scale = torch.ones((E, N, F // 128), dtype=torch.bfloat16, device="cuda")
    assert codes.numel() > 2 ** 31
    codes[E - 1] = 0x99  # code 9: the value 1
    gu = fp.W4Weight(torch.full((E, 2 * F, 16), 0x99, dtype=torch.uint8, device="cuda"),
                     torch.ones((E, 2 * F, 1), dtype=torch.bfloat16, device="cuda"), None, 32)
    dn = fp.W4Weight(codes, scale, None, 128)
    x = torch.zeros((1, 32), dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 8.0  # silu(8) * 8 = 63.98: 64 in bf16
    e = torch.full((1, 1), E - 1, dtype=torch.int32, device="cuda")
    y = fp.fp8_w4_experts(x, torch.ones((1, 1), device="cuda"), e, gu, dn)
    assert bool((y == 64.0 * F).all())


WIDE = [  # N, K: weights enough for the kernel of many tokens, ragged tiles and chunks of each group size
    (2064, 4128), (8192, 1056), (4112, 2080), (32768, 256)]


@pytest.mark.parametrize("N,K", WIDE)
@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (64, True), (128, False), (128, True)])
def test_many_tokens(fp, N, K, group, zero):
    w, v = weight(fp, (N, K), group, zero, N)
    v = v.cuda()
    for T in (17, 32, 33, 64, 65, 200):
        g = torch.Generator().manual_seed(T)
        x = torch.randn((T, K), generator=g).bfloat16().cuda()
        out = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
        y = fp.fp8_w4_linear(x, w, out=out[:T])
        want, bound = product(x.double(), v)
        off = (y.double() - want).abs()
        assert bool((off <= bound + want.abs() * UB + 1e-38).all()), (T, float((off - want.abs() * UB).max()))
        assert bool((out[T] == 7.0).all())
        if N % 32 == 0:
            h = fp.fp8_w4_gated(x, w, "gelu" if zero else "silu").double()
            want, bound = gated(x.double(), v, "gelu" if zero else "silu")
            assert bool(((h - want).abs() <= (bound + want.abs() * UB) * 1.01 + 1e-38).all())
    assert fp.fp8_get_device_status() == 0


@pytest.mark.parametrize("group,zero", [(32, True), (128, False)])
def test_many_tokens_an_expert(fp, group, zero):
    """Lists longer and shorter than a tile of tokens, an expert without a token, NaN in one token."""
    E, K, F, N, T, k = 5, 1056, 1024, 1040, 150, 2
    gu, vgu = weight(fp, (E, 2 * F, K), group, zero, 1)
    dn, vdn = weight(fp, (E, N, F), group, zero, 2)
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, K), generator=g).bfloat16()
    e = torch.randint(0, E - 1, (T, k), generator=g, dtype=torch.int32)
    e[:100] = torch.tensor([0, 2], dtype=torch.int32)
    e[torch.rand((T, k), generator=g) < 0.1] = -1
    w = torch.rand((T, k), generator=g)
    ws = fp.w4_experts_workspace(T, k, gu, dn).fill_(0xff)  # NaN wherever it is read as numbers
    y = fp.fp8_w4_experts(x.cuda(), w.cuda(), e.cuda(), gu, dn, ws=ws).cpu()
    want, bound = torch.zeros((T, N), dtype=torch.float64), torch.zeros((T, N), dtype=torch.float64)
    for i in range(E):
        t, j = (e == i).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        h, eh = gated(x.double()[t], vgu[i], "silu")
        eh = eh * 1.01 + h.abs() * UB * 1.01
        z, ez = product(h, vdn[i])
        ez = ez * (1 + UB) + eh @ vdn[i].abs().t()
        ww = w.double()[t, j][:, None]
        want.index_add_(0, t, ww * z)
        bound.index_add_(0, t, ww * (ez + z.abs() * (k + 2) * U))
    assert bool(((y.double() - want).abs() <= bound + want.abs() * UB + 1e-38).all())
    x2 = x.clone()
    x2[7, 3] = math.nan
    y2 = fp.fp8_w4_experts(x2.cuda(), w.cuda(), e.cuda(), gu, dn).cpu()
    keep = torch.arange(T) != 7
    assert torch.equal(y2[keep], y[keep]) and (bool(y2[7].isnan().all()) or bool((e[7] < 0).all()))
    assert fp.fp8_get_device_status() == 0


def test_many_tokens_in_a_graph(fp):
    w, _ = weight(fp, (4096, 2112), 64, True, 5)
    x = torch.randn((40, 2112), device="cuda").bfloat16()
    ws = fp.w4_workspace(w, 40)
    y = fp.fp8_w4_linear(x, w, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp.fp8_w4_linear(x, w, out=y, ws=ws)
    for _ in range(5):
        x.normal_()
        g.replay()
        assert torch.equal(y, fp.fp8_w4_linear(x, w))


@pytest.mark.parametrize("power", [-120, -100, 100, 115])
@pytest.mark.parametrize("group,zero", [(32, True), (128, False)])
def test_small_and_large_values(fp, power, group, zero):
    """Tokens near either end of bf16: besides the usual bound, a sum of a warp's 256
    terms is rounded at fp32's last denormal step 2^-149 at worst, 2^12 times smaller
    than the product, and the result at bf16's, 2^-133."""
    for N, K in ((64, 512), (16384, 512), (64, 8192)):
        w, v = weight(fp, (N, K), group, zero, N + K)
        for T in (1, 9, 40):
            x = (torch.randn((T, K), generator=torch.Generator().manual_seed(T)) * 2.0 ** power).bfloat16()
            y = fp.fp8_w4_linear(x.cuda(), w).cpu().double()
            want, bound = product(x.double(), v)
            bound = bound + K / 256 * 2.0 ** -136 + 2.0 ** -134 + K * 2.0 ** -149
            assert bool(((y - want).abs() <= bound + want.abs() * UB).all()), (N, K, T)


def experts_product(x, e, w, vgu, vdn, act):
    """fp8_w4_experts in 64 bits and its bound before the last rounding."""
    k = e.shape[1]
    want = torch.zeros((x.shape[0], vdn.shape[1]), dtype=torch.float64)
    bound = torch.zeros_like(want)
    for i in range(vgu.shape[0]):
        t, j = (e == i).nonzero(as_tuple=True)
        if t.numel():
            h, eh = gated(x.double()[t], vgu[i], act)
            eh = eh * 1.01 + h.abs() * UB * 1.01
            z, ez = product(h, vdn[i])
            ez = ez * (1 + UB) + eh @ vdn[i].abs().t()
            ww = w.double()[t, j][:, None]
            want.index_add_(0, t, ww * z)
            bound.index_add_(0, t, ww.abs() * (ez + z.abs() * (k + 2) * U))
    return want, bound


@pytest.mark.parametrize("T,E,k,K,F,N", [(40, 24, 2, 96, 32, 16), (9, 70, 3, 320, 96, 48), (130, 12, 2, 544, 256, 160),
                                         (50, 6, 3, 2048, 512, 256), (2, 1024, 4, 64, 32, 32)])
@pytest.mark.parametrize("kind", ["one", "last", "none", "steps", "twice"])
def test_experts_of_uneven_lists(fp, T, E, k, K, F, N, kind):
    """Lists far longer than others, empty ones between them, fewer items than blocks, the same
    expert twice in a token, and the workspace of another choice used again."""
    gu, vgu = weight(fp, (E, 2 * F, K), 64, True, E)
    dn, vdn = weight(fp, (E, N, F), 64, True, F)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, K), generator=g).bfloat16()
    w = torch.rand((T, k), generator=g)
    e = torch.full((T, k), -1, dtype=torch.int32)
    if kind == "one":
        e[:, 0] = E // 2
    elif kind == "last":
        e[:, k - 1] = E - 1
        e[0, 0] = 0
    elif kind == "steps":  # expert i has about twice the tokens of expert i + 2
        at = torch.rand((T, k), generator=g).log2().mul(-2).int()
        e = torch.where(at * 2 < E, at * 2, torch.tensor(-1, dtype=torch.int32)).contiguous()
    elif kind == "twice":
        e[:] = torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32)
    ws = fp.w4_experts_workspace(T, k, gu, dn).fill_(0xff)
    every = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    for choice in (e, every, e):
        y = fp.fp8_w4_experts(x.cuda(), w.cuda(), choice.cuda(), gu, dn, "gelu", ws=ws).cpu()
        want, bound = experts_product(x, choice, w, vgu, vdn, "gelu")
        assert bool(((y.double() - want).abs() <= bound + want.abs() * UB + 1e-38).all())



@pytest.mark.parametrize("N,K,T", [(2048, 512, 37), (512, 512, 700), (4096, 4096, 12), (1024, 1024, 90), (2080, 2048, 30),
                                   (48, 9216, 100)])
@pytest.mark.parametrize("group,zero", [(32, False), (64, True), (128, True)])
def test_blocks_of_few_tokens(fp, N, K, T, group, zero):
    """Small weights with more tokens than a block takes: blocks of tokens side by side, the last one short."""
    w, v = weight(fp, (N, K), group, zero, N + T)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).bfloat16()
    out = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = fp.fp8_w4_linear(x.cuda(), w, out=out[:T]).cpu().double()
    want, bound = product(x.double(), v)
    assert bool(((y - want).abs() <= bound + want.abs() * UB + 1e-38).all()) and bool((out[T] == 7.0).all())
    if N % 32 == 0:
        h = fp.fp8_w4_gated(x.cuda(), w, "silu").cpu().double()
        want, bound = gated(x.double(), v, "silu")
        assert bool(((h - want).abs() <= (bound + want.abs() * UB) * 1.01 + 1e-38).all())
