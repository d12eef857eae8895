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


PDL_CHILD = r"""
import hashlib
import torch
import fp8_mixed_precision_gb300 as fp
from fp8_mixed_precision_gb300 import synthetic as syn
from fp8_mixed_precision_gb300.gated_mlp import FP8GatedMLPStack

h = hashlib.sha256()
for recipe in ("block", "tensorwise"):
    m = FP8GatedMLPStack(512, 1024, 2, 1040, recipe, max_norm=0.1)
    xs = [syn.bf16_normal((1040, 512), 1.0, 42 + i, device="cuda") for i in range(2)]
    dys = [syn.bf16_normal((1040, 512), 1e-2, 44 + i, device="cuda") for i in range(2)]
    norm, grads = m.step(xs, dys)
    m.load()
    for t in [norm, *grads, m.decode(xs[0][:1]), m.decode(xs[0][:77])]:
        h.update(t.contiguous().view(torch.uint8).cpu().numpy().tobytes())
assert fp.fp8_get_device_status() == 0
print(h.hexdigest())
"""


def test_overlapped_and_plain_launches_give_the_same_bytes(tmp_path):
    """The launch mode is read once per process: two children, every kernel of
    the step and of decoding."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    script = tmp_path / "child.py"
    script.write_text(PDL_CHILD)
    out = []
    for pdl in ("0", "1"):
        env = dict(os.environ, FP8LIN_PDL=pdl, PYTHONPATH=root + os.pathsep + os.environ.get("PYTHONPATH", ""))
        r = subprocess.run([sys.executable, str(script)], cwd=root, env=env, capture_output=True, text=True,
                           timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        out.append(r.stdout.strip().splitlines()[-1])
    assert out[0] == out[1]


@pytest.mark.parametrize("recipe", ["block", "tensorwise"])
def test_a_step_replays_from_a_graph(fp, recipe):
    """Norm, gated feed-forward, linear and clipping captured in a CUDA graph and
    replayed on new inputs equal the same calls made one by one."""
    n, d, F = 160, 256, 384
    g = torch.Generator().manual_seed(3)
    x = torch.randn((n, d), generator=g).to(torch.bfloat16).cuda()
    dy = (torch.randn((n, F), generator=g) * 1e-2).to(torch.bfloat16).cuda()
    w = (torch.randn((2 * F, d), generator=g) * 0.05).to(torch.bfloat16).cuda()
    wn = torch.ones(d, device="cuda")
    cache = fp.WeightCache()
    h = cache.register(w, recipe)
    cache.begin_cycle()
    cache.get(h)
    ctx = fp.gated_context(recipe, n, d, F, "cuda")
    ws = fp.gated_workspace(recipe, n, d, F, "cuda")
    buf = fp.rmsnorm_buffers(n, d, "cuda", residual=False, rowwise=False, colwise=False, bf16=True)
    nws = fp.rmsnorm_workspace(n, d, "cuda")
    y, dx, dw = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((n, F), (n, d), (2 * F, d)))
    dxn, dwn = torch.empty_like(dx), torch.empty(d, device="cuda")
    acc = [torch.empty_like(dw), torch.empty_like(dwn)]
    clip = fp.GradClip([dw, dwn], acc)

    def step():
        o = fp.fp8_rmsnorm_fwd(x, wn, rowwise=False, colwise=False, bf16=True, out=buf)
        fp.fp8_gated_fwd(o["y"], cache, h, recipe, ws=ws, y=y, ctx=ctx)
        fp.fp8_gated_bwd(dy, ctx, cache, h, recipe, ws=ws, dx=dx, dw=dw)
        fp.fp8_rmsnorm_bwd(dx, x, o["rstd"], wn, dx=dxn, dw=dwn, ws=nws)
        clip.clip(0.01)

    step()  # loads every kernel
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn((n, d), generator=g).to(torch.bfloat16))
    step()
    want = [t.clone() for t in (y, dxn, *acc)]
    for t in (y, dxn, *acc):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (y, dxn, *acc)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("recipe", ["block", "tensorwise"])
def test_calls_on_another_stream_keep_their_scratch(fp, recipe):
    """Workspaces made inside a call on another stream are not handed to the
    current stream's allocations while that call still runs."""
    n, d, F = 700, 512, 640
    g = torch.Generator().manual_seed(9)
    x = torch.randn((n, d), generator=g).to(torch.bfloat16).cuda()
    dy = (torch.randn((n, F), generator=g) * 1e-2).to(torch.bfloat16).cuda()
    w = (torch.randn((2 * F, d), generator=g) * 0.05).to(torch.bfloat16).cuda()
    wn = torch.ones(d, device="cuda")
    rstd = torch.ones(n, device="cuda")
    cache = fp.WeightCache()
    h = cache.register(w, recipe)
    cache.begin_cycle()
    cache.get(h)

    def calls(stream):
        y, ctx = fp.fp8_gated_fwd(x, cache, h, recipe, stream=stream)
        junk(stream)
        dx, dw = fp.fp8_gated_bwd(dy, ctx, cache, h, recipe, stream=stream)
        junk(stream)
        dxn, dwn = fp.fp8_rmsnorm_bwd(dx, x, rstd, wn, stream=stream)
        junk(stream)
        keep.append(ctx)
        return y, dx, dw, dxn, dwn

    def junk(stream):
        if stream is not None:  # what the current stream allocates next is written at once
            for rows in (n, 4 * n, 16 * n):
                torch.full((rows, 2 * d), float("nan"), dtype=torch.bfloat16, device="cuda")
            stream.wait_stream(torch.cuda.current_stream())  # the next call's outputs may lie there

    keep = []
    want = calls(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        got = calls(s)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
