"""The norm, the gated feed-forward, the FP8 linear and clipping as one
training step and one decoded batch.

Against the same stack in 64 bits without any quantization: every FP8 operand
carries up to 2^-4 (E4M3) or 2^-3 (E5M2) of relative error per element, so the
chain of a few layers is held to 10% (outputs) and 35% (gradients) of the norm
only.  What is exact is held exactly: the same step with and without cached
weights, the clipped gradients' norm, decoding against training outputs.
"""
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


def _inputs(n, d, count, seed=1):
    g = torch.Generator().manual_seed(seed)
    xs = [torch.randn((n, d), generator=g).to(torch.bfloat16).cuda() for _ in range(count)]
    dys = [(torch.randn((n, d), generator=g) * 1e-2).to(torch.bfloat16).cuda() for _ in range(count)]
    return xs, dys


def _norm64(x, w):
    return x * (x.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * w


def _stack64(m, x, wgu, wd, wn):
    s, b = None, x
    for l in range(m.L):
        s = b if s is None else s + b
        gu = _norm64(s, wn[l]) @ wgu[l].t()
        b = (ref.act(gu[:, :m.F], m.act)[0] * gu[:, m.F:]) @ wd[l].t()
    return _norm64(s + b, wn[m.L])


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("recipe,act", [("block", "silu"), ("block", "gelu"), ("tensorwise", "silu")])
def test_step_follows_the_unquantized_stack(fp, recipe, act):
    from fp8_mixed_precision_gb300.gated_mlp import FP8GatedMLPStack
    n, d, ffn, layers = 272, 256, 384, 2
    m = FP8GatedMLPStack(d, ffn, layers, n, recipe, act, max_norm=1e30)
    xs, dys = _inputs(n, d, 2)
    norm, grads = m.step(xs, dys)
    P = [[t.double().requires_grad_() for t in ws] for ws in (m.wgu, m.wd, m.wn)]
    loss = 0
    for x, dy in zip(xs, dys):
        loss = loss + (_stack64(m, x.double(), *P) * dy.double()).sum()
    loss.backward()
    exact = [t.grad for ws in P for t in ws]
    for got, e in zip(grads, exact):
        assert _rel(got, e) < 0.35
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(norm) - want) < 1e-4 * want
    m.cache.begin_cycle()
    m.version += 1
    y, dx = m.microbatch(xs[0], dys[0])
    x = xs[0].double().requires_grad_()
    out = _stack64(m, x, *[[t.detach() for t in ws] for ws in P])
    (out * dys[0].double()).sum().backward()
    assert _rel(y, out.detach()) < 0.1
    assert _rel(dx, x.grad) < 0.35
    assert fp.fp8_get_device_status() == 0


@pytest.mark.parametrize("recipe", ["block", "tensorwise"])
def test_cached_weights_and_clipping(fp, recipe):
    from fp8_mixed_precision_gb300.gated_mlp import FP8GatedMLPStack
    n, d, ffn, layers = 128, 256, 256, 3
    xs, dys = _inputs(n, d, 3)
    runs = []
    for use_cache, max_norm in ((True, 1e30), (False, 1e30), (True, 0.25)):
        m = FP8GatedMLPStack(d, ffn, layers, n, recipe, max_norm=max_norm)
        norm, grads = m.step(xs, dys, use_cache=use_cache)
        runs.append((float(norm), [g.clone() for g in grads]))
    assert runs[0][0] == runs[1][0]
    assert all(torch.equal(a, b) for a, b in zip(runs[0][1], runs[1][1]))
    assert runs[2][0] == runs[0][0] > 0.25
    clipped = math.sqrt(sum(float(g.double().square().sum()) for g in runs[2][1]))
    assert abs(clipped - 0.25) < 1e-5
    coef = torch.tensor(0.25 / (runs[0][0] + 1e-6), dtype=torch.float64)
    for a, b in zip(runs[0][1], runs[2][1]):
        assert float((a.double() * coef - b.double()).abs().max()) <= 1e-6 * float(b.abs().max()) + 1e-30


@pytest.mark.parametrize("recipe", ["block", "tensorwise"])
@pytest.mark.parametrize("n", [1, 17, 160])
def test_decode_any_number_of_tokens(fp, recipe, n):
    """Under the block recipe a token's output depends on its own row only (each
    1x128 block is scaled by itself), so a decoded batch equals the rows of a
    larger one up to the order of fp32 sums (the few-token kernel splits K):
    one bf16 rounding may fall the other way at each of the chain's stages."""
    from fp8_mixed_precision_gb300.gated_mlp import FP8GatedMLPStack
    d, ffn, layers = 512, 768, 2
    m = FP8GatedMLPStack(d, ffn, layers, 16, recipe)
    m.load()
    x = _inputs(n, d, 1, seed=n)[0][0]
    y = m.decode(x)
    assert y.shape == (n, d)
    out = _stack64(m, x.double(), [w.double() for w in m.wgu], [w.double() for w in m.wd],
                   [w.double() for w in m.wn])
    assert _rel(y, out) < 0.1
    if recipe == "block":
        more = torch.cat([x, _inputs(40, d, 1, seed=99)[0][0]])
        assert _rel(m.decode(more)[:n], y.double()) < 2e-2


def test_example_runs(fp, capsys):
    from fp8_mixed_precision_gb300 import gated_mlp
    gated_mlp.main()
    assert "one token" in capsys.readouterr().out
