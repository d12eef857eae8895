"""Rows in the experts' order: the sort, gather, combine and their backward passes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative


@pytest.fixture(scope="module", autouse=True)
def fp():
    import fp8_mixed_precision_gb300 as fp
    fp.lib()
    return fp


def choices(T, k, E, seed, kind="random"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":            # every token takes the same expert, k times over
        return torch.full((T, k), E - 1, dtype=torch.int32)
    if kind == "none":
        return torch.full((T, k), -1, dtype=torch.int32)
    e = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if kind == "holes":
        e[torch.rand((T, k), generator=g) < 0.3] = -1
        e[torch.rand((T, k), generator=g) < 0.05] = E
        e[torch.rand((T, k), generator=g) < 0.05] = -2 ** 31
        e[T // 2:T // 2 + 3] = -1
    return e


def plain_order(e, E, align):
    """counts, offsets, position and the used part of order, as lists."""
    T, k = e.shape
    flat = e.reshape(-1).tolist()
    at = [[] for _ in range(E)]
    for s, x in enumerate(flat):
        if 0 <= x < E:
            at[x].append(s)
    offsets, position, order = [0], [-1] * (T * k), []
    for x in range(E):
        for i, s in enumerate(at[x]):
            position[s] = offsets[-1] + i
        rows = -(-len(at[x]) // align) * align
        order += at[x] + [-1] * (rows - len(at[x]))
        offsets.append(offsets[-1] + rows)
    return [len(a) for a in at], offsets, position, order


SIZES = [(1, 1, 1), (1, 8, 8), (3, 2, 5), (37, 4, 32), (64, 8, 256), (300, 3, 7), (1024, 2, 16), (1025, 2, 16),
         (5000, 6, 61), (70000, 2, 1024), (1, 1, 1024), (4097, 32, 3)]


@pytest.mark.parametrize("T,k,E", SIZES)
@pytest.mark.parametrize("align", [1, 16, 5])
@pytest.mark.parametrize("kind", ["random", "holes", "one", "none"])
def test_order(fp, T, k, E, align, kind):
    e = choices(T, k, E, T + k + E, kind)
    o = fp.fp8_expert_order(e.cuda(), E, align)
    counts, offsets, position, order = plain_order(e, E, align)
    assert o.counts.tolist() == counts and o.offsets.tolist() == offsets
    assert o.position.reshape(-1).tolist() == position
    assert o.rows >= offsets[-1] and o.order[:offsets[-1]].tolist() == order


def test_order_again(fp):
    """An order written again, rows past those in use left as they were; no tokens."""
    o = fp.fp8_expert_order(choices(50, 2, 8, 1).cuda(), 8, 16)
    o.order.fill_(77)
    e = choices(50, 2, 8, 2, "holes")
    p = fp.fp8_expert_order(e.cuda(), 8, 16, out=o)
    counts, offsets, position, order = plain_order(e, 8, 16)
    assert p is o and o.order.tolist() == order + [77] * (o.rows - len(order))
    z = fp.fp8_expert_order(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4)
    assert z.offsets.tolist() == [0] * 5 and z.counts.tolist() == [0] * 4 and z.rows == 0
    x = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    assert fp.fp8_expert_gather(x, z).shape == (0, 32) and fp.fp8_expert_combine(x, z).shape == (0, 32)


MOVES = [(1, 1, 1, 16), (1, 8, 8, 4096), (37, 4, 32, 4096), (61, 3, 5, 48), (130, 2, 16, 512), (9, 7, 4, 1040),
         (1000, 5, 11, 272), (5, 32, 40, 8192), (257, 2, 300, 1024)]


@pytest.mark.parametrize("T,k,E,C", MOVES)
@pytest.mark.parametrize("align", [1, 16])
@pytest.mark.parametrize("kind", ["random", "holes"])
def test_moves(fp, T, k, E, C, align, kind):
    e = choices(T, k, E, T + C, kind)
    o = fp.fp8_expert_order(e.cuda(), E, align)
    counts, offsets, position, order = plain_order(e, E, align)
    g = torch.Generator().manual_seed(C)

    def rnd(*shape):
        return torch.randn(shape, generator=g).bfloat16()
    x, z, dy = rnd(T, C), rnd(o.rows, C), rnd(T, C)
    w = torch.rand((T, k), generator=g)
    used = offsets[-1]
    row = torch.tensor(order, dtype=torch.long)
    real = row >= 0
    t_of = row.clamp(min=0) // k
    # gather: copies, zeros in the gaps, the rest untouched
    xs = torch.full((o.rows, C), 7.0, dtype=torch.bfloat16, device="cuda")
    assert fp.fp8_expert_gather(x.cuda(), o, out=xs) is xs
    want = torch.full((o.rows, C), 7.0, dtype=torch.bfloat16)
    want[:used] = torch.where(real[:, None], x[t_of], torch.zeros((), dtype=torch.bfloat16))
    assert torch.equal(xs.cpu(), want)
    # combine: k products and sums in fp32, one rounding to bf16
    pos = torch.tensor(position).view(T, k)
    zz = torch.where((pos >= 0)[..., None], z.double()[pos.clamp(min=0)], 0.0)
    for weights in (w, None):
        ww = torch.ones((T, k), dtype=torch.float64) if weights is None else w.double()
        y = fp.fp8_expert_combine(z.cuda(), o, None if weights is None else w.cuda())
        terms = zz * ww[..., None]
        bound = terms.abs().sum(1) * (k + 1) * U * 1.01 + terms.sum(1).abs() * UB + 1e-38
        assert bool(((y.cpu().double() - terms.sum(1)).abs() <= bound * (1 + UB)).all())
    # backward: one product and one rounding; dot products of C terms in fp32
    dz = torch.full((o.rows, C), 7.0, dtype=torch.bfloat16, device="cuda")
    got, dw = fp.fp8_expert_combine_bwd(dy.cuda(), z.cuda(), o, w.cuda(), dz=dz)
    assert got is dz
    exact = torch.where(real[:, None], dy.double()[t_of] * w.double().view(-1)[row.clamp(min=0)][:, None], 0.0)
    off = (dz[:used].cpu().double() - exact).abs()
    assert bool((off <= exact.abs() * (UB + 2 * U) + 1e-38).all())
    assert bool((dz[used:] == 7.0).all()) and bool((dz[:used].cpu()[~real] == 0).all())
    prod = zz * dy.double()[:, None]
    assert bool(((dw.cpu().double() - prod.sum(2)).abs() <= prod.abs().sum(2) * (C / 32 + 40) * U + 1e-38).all())
    assert bool((dw.cpu()[pos < 0] == 0).all())


def test_nan_weight_shows(fp):
    """A token whose routing failed (experts -1, weights NaN) gives NaN, other empty slots nothing."""
    e = torch.tensor([[-1, -1], [0, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[float("nan")] * 2, [1.0, 0.0], [0.0, 0.0]], device="cuda")
    o = fp.fp8_expert_order(e, 2)
    z = torch.ones((o.rows, 16), dtype=torch.bfloat16, device="cuda")
    y = fp.fp8_expert_combine(z, o, w)
    assert bool(y[0].isnan().all()) and bool((y[1] == 1).all()) and bool((y[2] == 0).all())


def test_streams_and_graph(fp):
    T, k, E, C = 300, 2, 8, 512
    x = torch.randn((T, C), device="cuda").bfloat16()
    e = choices(T, k, E, 3).cuda()
    w = torch.rand((T, k), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = fp.fp8_expert_order(e, E, 16, stream=s)
    y = fp.fp8_expert_combine(fp.fp8_expert_gather(x, o, stream=s), o, w, stream=s)
    s.synchronize()
    o2 = fp.fp8_expert_order(e, E, 16)
    xs = torch.zeros((o2.rows, C), dtype=torch.bfloat16, device="cuda")
    y2 = fp.fp8_expert_combine(fp.fp8_expert_gather(x, o2, out=xs), o2, w)
    assert torch.equal(y, y2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp.fp8_expert_order(e, E, 16, out=o2)
        fp.fp8_expert_gather(x, o2, out=xs)
        fp.fp8_expert_combine(xs, o2, w, out=y2)
    for seed in (5, 6):
        e.copy_(choices(T, k, E, seed, "holes"))
        x.normal_()
        g.replay()
        o3 = fp.fp8_expert_order(e, E, 16)
        assert torch.equal(y2, fp.fp8_expert_combine(fp.fp8_expert_gather(x, o3), o3, w))


def test_rows_past_32_bits(fp):
    """Elements past 2^31 of the row buffers."""
    C, T = 16384, 70000
    k = 2
    e = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    e[:, 1] = 1
    o = fp.fp8_expert_order(e, 2)
    x = torch.randn((T, C), device="cuda", dtype=torch.bfloat16)
    xs = fp.fp8_expert_gather(x, o)
    assert xs.numel() > 2 ** 31 and torch.equal(xs[:T], x) and torch.equal(xs[T:], x)
    w = torch.ones((T, k), device="cuda")
    assert torch.equal(fp.fp8_expert_combine(xs, o, w), x * 2)
    dz, dw = fp.fp8_expert_combine_bwd(x, xs, o, w)
    assert torch.equal(dz, xs) and torch.equal(dw[:, 0], dw[:, 1])
    want = x[-1].double().square().sum()
    assert abs(float(dw[-1, 1]) - float(want)) <= float(want) * (C / 32 + 40) * U


@pytest.mark.parametrize("T,k,E,C", [(19, 2, 6, 2048), (33, 1, 4, 1552), (21, 2, 5, 4112), (40, 1, 3, 8192), (50, 3, 7, 1936)])
@pytest.mark.parametrize("kind", ["random", "holes"])
def test_moves_of_other_row_lengths(fp, T, k, E, C, kind):
    test_moves(fp, T, k, E, C, 16, kind)
