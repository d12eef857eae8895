"""Routing to experts against a plain statement in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24  # half a step of fp32, relative
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def fp():
    import fp8_mixed_precision_gb300 as fp
    fp.lib()
    return fp


def scores(l, score):
    """s of one token's logits (a list of floats); None where it is NaN."""
    if any(math.isnan(v) for v in l) or (score == "softmax" and INF in l):
        return None
    if score == "sigmoid":
        return [0.0 if v == -INF else 1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in l]
    m = max(l)
    if m == -INF:
        return [0.0] * len(l)
    p = [math.exp(v - m) for v in l]
    return [v / math.fsum(p) for v in p]


def choose(l, k, score, bias, groups, kept, top):
    """Experts of one token, from the definition: fp64 throughout."""
    s = scores(l, score)
    if s is None:
        return None
    E = len(l)
    c = [-INF if l[e] == -INF else s[e] + (bias[e] if bias else 0.0) for e in range(E)]
    if any(math.isnan(v) for v in c):
        return None
    per = E // groups
    if groups > 1:
        def value(g):
            best = sorted((c[e] for e in range(g * per, (g + 1) * per)), reverse=True)[:top]
            best = [v for v in best if v > -INF]
            return sum(best) if best else -INF
        order = sorted((g for g in range(groups) if value(g) > -INF), key=lambda g: (-value(g), g))[:kept]
        c = [c[e] if e // per in order else -INF for e in range(E)]
    # without a bias the scores are in the order of the logits, rounded or not
    rank = (lambda e: (-c[e], -l[e], e)) if not bias else (lambda e: (-c[e], e))
    best = sorted((e for e in range(E) if c[e] > -INF), key=rank)[:k]
    return best + [-1] * (k - len(best))


def weights_of(l, experts, score, renorm, scale):
    s = scores(l, score)
    u = [0.0 if e < 0 else s[e] for e in experts]
    total = math.fsum(u)
    if renorm:
        if total == 0.0:  # all underflow: the ratios of the logarithms
            g = [-INF if e < 0 else l[e] for e in experts]
            m = max(g)
            u = [0.0 if v == -INF else math.exp(v - m) for v in g] if m > -INF else u
            total = math.fsum(u) or 1.0
        u = [v / total for v in u]
    return [v * scale for v in u]


def check(fp, logits, k, score="softmax", bias=None, groups=1, kept=None, top=1, renorm=True, scale=1.0):
    kept = groups if kept is None else kept
    T, E = logits.shape
    w, e = fp.fp8_route_fwd(logits.cuda(), k, score, None if bias is None else bias.cuda(), groups, kept, top, renorm,
                            scale)
    ll = logits.double().tolist()
    bl = None if bias is None else bias.double().tolist()
    we, ee = w.double().cpu().tolist(), e.cpu().tolist()
    # w: exponentials (2 ulp each and the rounding of their argument, at most
    # |l - m| U where the value itself is e^-|l - m|), sums of E terms, a division
    rel = (E / 8 + 40) * U
    for t in range(T):
        want = choose(ll[t], k, score, bl, groups, kept, top)
        if want is None:
            assert ee[t] == [-1] * k and all(math.isnan(v) for v in we[t]), t
            continue
        assert ee[t] == want, (t, ee[t], want)
        for a, b in zip(we[t], weights_of(ll[t], want, score, renorm, scale)):
            assert abs(a - b) <= rel * b + 100 * U * b + 1e-37 * scale, (t, a, b)
    return w, e


CASES = [  # T, E, k, score, bias, groups, kept, top, renorm, scale
    (1, 1, 1, "softmax", False, 1, 1, 1, True, 1.0),
    (5, 2, 2, "sigmoid", True, 1, 1, 1, False, 1.0),
    (33, 7, 3, "softmax", False, 1, 1, 1, True, 2.0),
    (17, 32, 8, "sigmoid", True, 4, 2, 2, True, 1.0),
    (17, 32, 9, "sigmoid", True, 4, 2, 2, True, 1.0),
    (9, 32, 32, "softmax", True, 32, 32, 1, True, 1.0),
    (19, 48, 5, "softmax", True, 12, 5, 2, False, 1.5),
    (50, 64, 8, "softmax", False, 1, 1, 1, True, 1.0),
    (31, 64, 16, "softmax", False, 8, 3, 2, True, 1.0),
    (64, 128, 8, "softmax", True, 1, 1, 1, False, 1.0),
    (29, 129, 8, "sigmoid", False, 3, 2, 1, True, 1.0),
    (61, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (21, 510, 6, "softmax", True, 5, 2, 2, True, 1.0),
    (23, 512, 12, "softmax", False, 1, 1, 1, False, 1.0),
    (11, 1021, 32, "sigmoid", True, 1, 1, 1, True, 1.0),
    (13, 1024, 10, "softmax", True, 32, 4, 2, False, 1.0),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,score,bias,groups,kept,top,renorm,scale", CASES)
def test_forward(fp, dtype, T, E, k, score, bias, groups, kept, top, renorm, scale):
    g = torch.Generator().manual_seed(E * 7 + T)
    logits = torch.randn((T, E), generator=g).to(dtype)
    b = 0.1 * torch.randn(E, generator=g) if bias else None
    check(fp, logits, k, score, b, groups, kept, top, renorm, scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 1), (4, 2)])
def test_masks(fp, score, bias, groups, top):
    """Rows without candidates, with fewer than k, in few groups; the type's lowest value; NaN and infinities."""
    E, k = 32, 6
    g = torch.Generator().manual_seed(3)
    l = torch.randn((12, E), generator=g)
    l[0] = -INF
    l[1, 3:] = -INF                # fewer candidates than slots
    l[2, : E - 1] = -INF
    l[3, 8:16] = -INF              # a whole group
    l[4, 1::2] = -INF
    l[5, 4:] = torch.finfo(torch.float32).min
    l[6] = torch.finfo(torch.float32).min
    l[7, 5] = math.nan
    l[8, 9] = INF
    l[9] = -120.0 + l[9]           # scores below fp32's range
    l[10, 1:] = -INF
    l[10, 0] = -INF
    b = 0.1 * torch.randn(E, generator=g) if bias else None
    if bias:
        b[7] = -INF
        b[11] = INF
    if bias and score == "softmax":
        l[8, 9] = 1.0
    kept = 4 if groups == 4 else 1
    for renorm in (True, False):
        check(fp, l, k, score, b, groups, kept, top, renorm)


def test_nan_bias(fp):
    b = torch.zeros(16)
    b[3] = math.nan
    w, e = check(fp, torch.randn((3, 16)), 2, "sigmoid", b)
    assert bool((e == -1).all()) and bool(w.isnan().all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,groups,kept,top", [(16, 1, 1, 1), (64, 8, 3, 2), (256, 8, 2, 1)])
def test_ties(fp, dtype, E, groups, kept, top):
    """Equal logits, equal scores with and without a bias: the lowest index."""
    g = torch.Generator().manual_seed(E)
    l = torch.randint(-2, 3, (40, E), generator=g).to(dtype)
    for bias in (None, torch.zeros(E), torch.randint(0, 2, (E,), generator=g).float() / 4):
        for score in ("softmax", "sigmoid"):
            check(fp, l, 5, score, bias, groups, kept, top)


def test_close_scores(fp):
    """Scores that fp32 cannot tell apart, in every place of the order."""
    E, k, T = 64, 8, 64
    g = torch.Generator().manual_seed(5)
    l = torch.randn((T, E), generator=g)
    b = torch.empty(E)
    b.uniform_(-0.05, 0.05, generator=g)
    # sigmoid(l) + b nearly equal for neighbours: the logits are shifted to undo the bias
    base = torch.linspace(0.3, 0.6, E // 4, dtype=torch.float64).repeat_interleave(4)
    for t in range(T):
        noise = torch.rand(E, generator=g, dtype=torch.float64) * 4e-8
        s = base[torch.randperm(E, generator=g)] + noise - b.double()
        l[t] = torch.log(s / (1 - s)).float()
    check(fp, l, k, "sigmoid", b)
    check(fp, l, k, "sigmoid", b, 8, 3, 2)
    check(fp, l, k, "softmax", b * 1e-7)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,score,bias,groups,kept,top,renorm,scale", CASES)
def test_backward(fp, dtype, T, E, k, score, bias, groups, kept, top, renorm, scale):
    g = torch.Generator().manual_seed(E + T)
    logits = torch.randn((T, E), generator=g).to(dtype)
    if E > k:
        logits[T // 2, E // 2:] = -INF
    logits[T - 1] = -INF
    b = 0.1 * torch.randn(E, generator=g) if bias else None
    kw = dict(score=score, renormalize=renorm, scale=scale)
    dev = logits.cuda()
    w, e = fp.fp8_route_fwd(dev, k, bias=None if b is None else b.cuda(), groups=groups, groups_kept=kept,
                            group_top=top, **kw)
    dw = torch.randn((T, k), generator=g)
    d = fp.fp8_route_bwd(dw.cuda(), dev, w, e, **kw)
    l = logits.double()
    ee = e.cpu().long()
    some = (ee >= 0).double()
    p = torch.sigmoid(l) if score == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    p = torch.where(l == -INF, 0.0, p)
    pc = p.gather(1, ee.clamp(min=0)) * some
    total = pc.sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    gr = dw.double() * scale
    u = pc / total if renorm else pc
    dp = (gr - (gr * u).sum(1, keepdim=True)) / total if renorm else gr
    full = torch.zeros_like(p).scatter_add_(1, ee.clamp(min=0), dp * some)
    want = full * p * (1 - p) if score == "sigmoid" else p * (full - (full * p).sum(1, keepdim=True))
    # every term is a product of factors within (E / 8 + 60) U, and they cancel
    # in the difference: the bound counts their magnitudes
    size = (full.abs() + (dp * some * pc).abs().sum(1, keepdim=True) + (gr * u).abs().sum(1, keepdim=True) / total
            * (full != 0)) * p
    out = 2.0 ** -8 if dtype == torch.bfloat16 else U
    bound = size * (E / 4 + 120) * U + want.abs() * out + 1e-38
    off = (d.double().cpu() - want).abs()
    assert d.dtype == dtype and bool((off <= bound).all()), float((off / bound).max())
    assert bool((d[T - 1] == 0).all())
    assert bool((d.cpu()[l == -INF] == 0).all())


def test_backward_by_differences(fp):
    T, E, k = 4, 24, 4
    g = torch.Generator().manual_seed(9)
    l = torch.randn((T, E), generator=g)
    dw = torch.randn((T, k), generator=g)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            kw = dict(score=score, renormalize=renorm, scale=1.5)
            w, e = fp.fp8_route_fwd(l.cuda(), k, **kw)
            d = fp.fp8_route_bwd(dw.cuda(), l.cuda(), w, e, **kw).cpu()
            ee = e.cpu().tolist()
            h = 1e-5  # error of the difference: h^2 / 6 times a third derivative of order one

            def loss(t, i, step):
                x = l[t].double().tolist()
                x[i] += step
                return math.fsum(a * b for a, b in zip(weights_of(x, ee[t], score, renorm, 1.5), dw[t].tolist()))
            for t in range(T):
                for i in range(E):
                    want = (loss(t, i, h) - loss(t, i, -h)) / (2 * h)
                    assert abs(float(d[t, i]) - want) < 1e-6


def test_views_streams_graph(fp):
    """Rows off the vectors' boundary, another stream, and a replayed graph on new values."""
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.randn((9 * 24 + 1,), device="cuda").to(dtype)
        l = base[1:].view(9, 24)
        w, e = fp.fp8_route_fwd(l, 4)
        w2, e2 = fp.fp8_route_fwd(l.clone(), 4)
        assert torch.equal(w, w2) and torch.equal(e, e2)
        d = fp.fp8_route_bwd(torch.ones_like(w), l, w, e)
        assert torch.equal(d, fp.fp8_route_bwd(torch.ones_like(w), l.clone(), w, e))
    s = torch.cuda.Stream()
    l = torch.randn((40, 64), device="cuda")
    torch.cuda.synchronize()
    w, e = fp.fp8_route_fwd(l, 4, stream=s)
    s.synchronize()
    want = fp.fp8_route_fwd(l, 4)
    assert torch.equal(w, want[0]) and torch.equal(e, want[1])
    out = (torch.empty_like(w), torch.empty_like(e))
    d = torch.empty_like(l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp.fp8_route_fwd(l, 4, out=out)
        fp.fp8_route_bwd(out[0], l, *out, out=d)
    for _ in range(3):
        l.copy_(torch.randn((40, 64)))
        g.replay()
        want = fp.fp8_route_fwd(l, 4)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert torch.equal(d, fp.fp8_route_bwd(want[0], l, *want))


def test_many_tokens(fp):
    """More blocks than the GPU holds, the last one part full; the same bits on each call."""
    T, E, k = 100003, 40, 5
    l = torch.randn((T, E), device="cuda")
    w, e = fp.fp8_route_fwd(l, k)
    v, i = l.sort(dim=1, descending=True, stable=True)
    assert torch.equal(e.long(), i[:, :k])
    assert float((w.double() - torch.softmax(v[:, :k].double(), 1)).abs().max()) < 64 * U
    w2, e2 = fp.fp8_route_fwd(l, k)
    assert torch.equal(w, w2) and torch.equal(e, e2)


def reference(l, k, score, bias, groups, kept, top, renorm, scale):
    """weights and experts of many tokens, in fp64 on the GPU (no ties but of equal logits and biases)."""
    l = l.double()
    masked = l == -INF
    p = torch.sigmoid(l) if score == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    c = torch.where(masked, -INF, p if bias is None else p + bias.double())
    T, E = l.shape
    if groups > 1:
        g = c.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :top]
        v = torch.where(g == -INF, 0.0, g).sum(2)
        v = torch.where(g[:, :, 0] == -INF, -INF, v)
        keep = v.sort(dim=1, descending=True, stable=True).indices[:, :kept]
        out = torch.ones((T, groups), dtype=torch.bool, device=l.device).scatter_(1, keep, False)
        c = torch.where(out.repeat_interleave(E // groups, 1), -INF, c)
    v, e = c.sort(dim=1, descending=True, stable=True)
    v, e = v[:, :k], e[:, :k]
    e = torch.where(v == -INF, -1, e)
    w = torch.where(e < 0, 0.0, p.gather(1, e.clamp(min=0)))
    if renorm:
        w = w / torch.where(w.sum(1, keepdim=True) > 0, w.sum(1, keepdim=True), 1.0)
    return w * scale, e.int()


MANY = [  # E, k, score, bias, groups, kept, top, renorm
    (32, 8, "softmax", False, 1, 1, 1, False), (31, 3, "sigmoid", False, 1, 1, 1, True),
    (64, 8, "softmax", True, 1, 1, 1, True), (60, 7, "softmax", False, 4, 2, 2, True),
    (128, 8, "softmax", False, 1, 1, 1, False), (125, 6, "sigmoid", True, 5, 3, 2, True),
    (128, 12, "softmax", False, 8, 3, 1, True), (200, 9, "softmax", False, 1, 1, 1, False),
    (256, 16, "sigmoid", False, 8, 4, 2, False), (256, 6, "sigmoid", True, 8, 3, 2, True),
    (256, 17, "softmax", False, 1, 1, 1, True), (512, 8, "softmax", True, 16, 4, 1, False),
    (130, 24, "sigmoid", True, 1, 1, 1, True), (1000, 10, "softmax", False, 1, 1, 1, True)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k,score,bias,groups,kept,top,renorm", MANY)
def test_many_tokens_every_way(fp, dtype, E, k, score, bias, groups, kept, top, renorm):
    """Enough tokens for few lanes to each one, forward and backward, the last block part full."""
    T = 6001
    g = torch.Generator(device="cuda").manual_seed(E + k)
    l = torch.randn((T, E), generator=g, device="cuda").to(dtype)
    l[5] = -INF
    l[T - 1, k // 2:] = -INF
    b = 0.1 * torch.randn(E, generator=g, device="cuda") if bias else None
    kw = dict(score=score, renormalize=renorm, scale=1.5)
    w, e = fp.fp8_route_fwd(l, k, bias=b, groups=groups, groups_kept=kept, group_top=top, **kw)
    ww, ee = reference(l, k, score, b, groups, kept, top, renorm, 1.5)
    assert torch.equal(e, ee)
    assert bool(((w.double() - ww).abs() <= ww * (E / 8 + 140) * U + 1e-37).all())
    dw = torch.randn((T, k), generator=g, device="cuda")
    d = fp.fp8_route_bwd(dw, l, w, e, **kw)
    # the same tokens few at a time take 32 lanes each: other orders of the same sums
    few = torch.cat([fp.fp8_route_bwd(dw[i:i + 1000], l[i:i + 1000], w[i:i + 1000], e[i:i + 1000], **kw)
                     for i in range(0, T, 1000)])
    p = (torch.sigmoid(l.double()) if score == "sigmoid" else torch.nan_to_num(torch.softmax(l.double(), 1)))
    gr = dw.double().abs() * w.double().abs()
    size = torch.zeros_like(p).scatter_add_(1, ee.clamp(min=0).long(), gr + w.double() * gr.sum(1, keepdim=True))
    size = size + p * gr.sum(1, keepdim=True)
    out = 2.0 ** -8 if dtype == torch.bfloat16 else U
    assert bool(((d.double() - few.double()).abs() <= 2 * (size * (E / 4 + 120) * U + d.double().abs() * out) + 1e-37).all())
    assert bool((d[5] == 0).all())


def test_backward_of_one_expert_named_twice(fp):
    """Rows that the forward pass does not make: both slots count."""
    for T in (3, 6000):
        l = torch.randn((T, 16), device="cuda")
        e = torch.zeros((T, 4), dtype=torch.int32, device="cuda")
        e[:, 2] = 5
        e[:, 3] = -1
        w = torch.rand((T, 4), device="cuda")
        dw = torch.randn((T, 4), device="cuda")
        d = fp.fp8_route_bwd(dw, l, w, e, score="sigmoid", renormalize=False)
        a = (dw * w).double() * torch.sigmoid(-l.double().gather(1, e.clamp(min=0).long()))
        want = torch.zeros((T, 16), dtype=torch.float64, device="cuda")
        want[:, 0] = a[:, 0] + a[:, 1]
        want[:, 5] = a[:, 2]
        assert bool(((d.double() - want).abs() <= 16 * U * (a.abs().sum(1, keepdim=True))).all())
