"""Routing, rows in the experts' order, the FP8 gated feed-forward and linear on
each expert's rows, and decoding on 4-bit weights, together.

Against the same stack in 64 bits on the experts that the run chose.  The
training pass is unquantized there, and FP8 operands carry up to 2^-4 (E4M3) or
2^-3 (E5M2) per element, so the chain is held to 10% (output) and 35% (gradients)
of the norm only; decoding is held to the 4-bit weights' own values, its router
alone in FP8."""
import math

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


def _norm64(x, w):
    return x * (x.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * w


def _mlp64(x, gu, d, act):
    F = d.shape[1]
    y = x @ gu.t()
    return (ref.act(y[:, :F], act)[0] * y[:, F:]) @ d.t()


def _stack64(m, x, experts, wr, wgu, wd, wn):
    s, b = None, x
    for l in range(m.L):
        s = b if s is None else s + b
        xn = _norm64(s, wn[l])
        e = experts[l].long()
        logits = xn @ wr[l].t()
        p = torch.softmax(logits, 1) if m.score == "softmax" else torch.sigmoid(logits)
        p = p.gather(1, e)
        w = p / p.sum(1, keepdim=True)
        b = torch.zeros_like(x)
        for i in range(m.E):
            t, j = (e == i).nonzero(as_tuple=True)
            if t.numel():
                b = b.index_add(0, t, _mlp64(xn[t], wgu[l][i], wd[l][i], m.act) * w[t, j][:, None])
    return _norm64(s + b, wn[m.L])


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def _inputs(n, d, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, d), generator=g).bfloat16().cuda(),
            (torch.randn((n, d), generator=g) * 1e-2).bfloat16().cuda())


@pytest.mark.parametrize("recipe,score,act", [("block", "softmax", "silu"), ("tensorwise", "sigmoid", "gelu")])
def test_step_follows_the_unquantized_stack(fp, recipe, score, act):
    from fp8_mixed_precision_gb300.expert_mlp import FP8ExpertMLPStack
    n, d, ffn, layers, E, k = 272, 256, 128, 2, 16, 3
    m = FP8ExpertMLPStack(d, ffn, layers, n, E, k, recipe, act, score, max_norm=1e30)
    x, dy = _inputs(n, d)
    norm, grads = m.step([x], [dy])
    got = [g.clone() for g in grads]
    assert all(int(c.sum()) == n * k for c in m.counts)
    m.cache.begin_cycle()
    m.version += 1
    y, dx, experts = m.microbatch(x, dy)
    P = [[t.double().requires_grad_() for t in ws] for ws in (m.wr, m.wgu, m.wd, m.wn)]
    xd = x.double().requires_grad_()
    out = _stack64(m, xd, experts, *P)
    (out * dy.double()).sum().backward()
    assert _rel(y, out.detach()) < 0.1
    assert _rel(dx, xd.grad) < 0.35
    exact = [t.grad for ws in P for t in ws]
    for a, e in zip(got, exact):
        assert _rel(a, e) < 0.35
    want = math.sqrt(sum(float(g.double().square().sum()) for g in got))
    assert abs(float(norm) - want) < 1e-4 * want
    assert fp.fp8_get_device_status() == 0


def test_steps_are_alike_and_balance_moves(fp):
    """The same step twice gives the same bytes, with and without cached weights; an
    expert with fewer tokens than the mean gains bias, one with more loses it."""
    from fp8_mixed_precision_gb300.expert_mlp import FP8ExpertMLPStack
    m = FP8ExpertMLPStack(256, 128, 1, 128, 16, 2, max_norm=1e30)
    x, dy = _inputs(128, 256, 5)
    runs = []
    for use_cache in (True, True, False):
        norm, grads = m.step([x, x], [dy, dy], use_cache=use_cache)
        runs.append((float(norm), [g.clone() for g in grads]))
    for norm, grads in runs[1:]:
        assert norm == runs[0][0] and all(torch.equal(a, b) for a, b in zip(runs[0][1], grads))
    m.balance(0.5)
    n = m.counts[0].float()
    assert torch.equal(m.bias[0], 0.5 * torch.sign(n.mean() - n))


@pytest.mark.parametrize("group,zero", [(128, False), (32, True)])
@pytest.mark.parametrize("n", [1, 17, 40])
def test_decode(fp, group, zero, n):
    from fp8_mixed_precision_gb300.expert_mlp import FP8ExpertMLPStack
    m = FP8ExpertMLPStack(512, 256, 1, 16, 16, 2)
    m.load(group, zero)
    x, _ = _inputs(n, 512, n)
    y = m.decode(x)

    def values(w):
        q = torch.stack((w.codes & 15, w.codes >> 4), -1).flatten(-2).double()
        at = torch.arange(w.K, device="cuda") // w.group
        return (q - (8.0 if w.zero is None else w.zero.double()[..., at])) * w.scale.double()[..., at]

    # the routing that decode() makes, from the same calls
    o = fp.fp8_rmsnorm_fwd(x, m.wn[0], rowwise=False, colwise=False, bf16=True)
    padded = torch.zeros((-(-n // 16) * 16, 512), dtype=torch.bfloat16, device="cuda")
    padded[:n] = o["y"]
    logits, _ = fp.fp8_linear_fwd(padded, m.cache, m.hr[0], m.recipe)
    w, e = fp.fp8_route_fwd(logits[:n], m.k, bias=m.bias[0])
    gu, dn = (values(t) for t in m.w4[0])
    b = torch.zeros((n, 512), dtype=torch.float64, device="cuda")
    for i in range(m.E):
        t, j = (e == i).nonzero(as_tuple=True)
        if t.numel():
            b.index_add_(0, t, _mlp64(o["y"].double()[t], gu[i], dn[i], m.act) * w[t, j].double()[:, None])
    out = _norm64(x.double() + b, m.wn[0].double())
    # roundings to bf16: the hidden values, the branch, the stream and the output,
    # each at most 2^-8 of its element
    assert _rel(y, out) < 4 * 2.0 ** -8
    assert fp.fp8_get_device_status() == 0


def test_example_runs(fp, capsys):
    from fp8_mixed_precision_gb300 import expert_mlp
    expert_mlp.main()
    assert "one token" in capsys.readouterr().out


def test_shared_use_on_two_streams(fp):
    """Decoding steps on two streams at once, each with its own buffers, give the bytes of one after the other."""
    from fp8_mixed_precision_gb300.expert_mlp import FP8ExpertMLPStack
    m = FP8ExpertMLPStack(512, 256, 1, 16, 16, 2)
    m.load(64)
    gu, dn = m.w4[0]
    xs = [_inputs(24, 512, s)[0] for s in (3, 4)]
    logits = [torch.randn((24, 16), device="cuda") for _ in xs]
    torch.cuda.synchronize()

    def run(i, stream):
        w, e = fp.fp8_route_fwd(logits[i], 2, stream=stream)
        return fp.fp8_w4_experts(xs[i], w, e, gu, dn, stream=stream)
    want = [run(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        got = [run(i, s) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
