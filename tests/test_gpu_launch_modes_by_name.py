"""Overlapped (programmatic dependent) and plain launches give the same bytes, output by
output: every kernel family, the norm's, the gated feed-forward's, the routing's, the
rows' and the 4-bit products' among them, run twice in each of two child processes,
FP8LIN_PDL=0 and FP8LIN_PDL=1, and each output's SHA-256 is kept under its name.  A name
that differs between the two passes of one process is a result that is not repeatable; one
that differs between the processes alone is a kernel that does not wait for the one before it."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))

CHILD = r'''
import hashlib, json
import torch
import fp8_mixed_precision_gb300 as fp
from fp8_mixed_precision_gb300 import synthetic as syn
from fp8_mixed_precision_gb300.mlp import FP8MLPStack

dev = "cuda"
names, sums = [], []


def add(name, *ts):
    for i, t in enumerate(ts):
        if t is not None:
            names.append(f"{name} {i}")
            sums.append(hashlib.sha256(t.contiguous().view(torch.uint8).cpu().numpy().tobytes()).hexdigest())


def normal(shape, std, seed):
    return syn.bf16_normal(shape, std, seed, device=dev)


def f32(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dev)


LINEAR = [(N, K, O, *syn.linear_inputs(N, K, O, device=dev, layer=i))
          for i, (N, K, O) in enumerate([(8192, 512, 2048), (16384, 512, 512), (8192, 512, 8192)])]
XS = [normal((4096, 512), 1.0, 42 + m) for m in range(2)]
DYS = [normal((4096, 512), 1e-3, 44 + m) for m in range(2)]
XD = [normal((2048, 1024), 1.0, 50 + s) for s in range(3)]
WG = normal((2 * 768, 512), 0.02, 60)
LOGITS = f32((5003, 64), 61)
BIAS = f32((64,), 62) * 0.05
DW = f32((5003, 6), 63)
ROWS, DROWS = normal((5003, 512), 1.0, 64), normal((5003, 512), 1e-3, 65)
W4 = [normal(s, 0.02, 70 + i) for i, s in enumerate([(2048, 512), (4096, 8192), (4096, 2048)])]
GU, DN = normal((8, 2 * 1024, 1024), 0.02, 80), normal((8, 1024, 1024), 0.02, 81)
GRADS = [normal((300, 512), 1.0, 90), normal((77, 16), 10.0, 91)]


def sequence():
    for N, K, O, x, w, dy in LINEAR:
        cache = fp.WeightCache()
        h = cache.register(w, "tensorwise")
        cache.begin_cycle()
        cache.get(h, 1, True)
        y, ctx = fp.fp8_linear_fwd(x, cache, h, "tensorwise")
        add(f"tensorwise linear {N} {K} {O}: y, dx, dw", y, *fp.fp8_linear_bwd(dy, ctx, cache, h, "tensorwise"))
    for fused in (False, True):
        st = FP8MLPStack(512, 2048, 2, 4096, "block", fused=fused)
        for m, (y, dx) in enumerate(st.step(XS, DYS, use_cache=True)):
            add(f"block stack, fused {fused}, microbatch {m}: y, dx", y, dx)
        add(f"block stack, fused {fused}: dw1, dw2", *st.dw1, *st.dw2)
    hist = torch.zeros(16, dtype=torch.float32, device=dev)
    for s in range(3):
        q = fp.fp8_quantize_delayed(XD[s], "act", hist, s)
        add(f"delayed scaling, step {s}", q["row"], q["col"], q["scale"], q["scale_inv"], hist)
    ones = torch.ones(512, device=dev)
    for recipe in ("tensorwise", "block"):
        cache = fp.WeightCache()
        h = cache.register(WG, recipe)
        cache.begin_cycle()
        cache.get(h, 1)
        for n in (1, 37, 1000):
            o = fp.fp8_rmsnorm_fwd(ROWS[:n], ones, residual=DROWS[:n], bf16=True)
            add(f"norm of {n}", o["r"], o["y"], o["row"], o["rstd"])
            y, ctx = fp.fp8_gated_fwd(o["y"], cache, h, recipe)
            dx, dw = fp.fp8_gated_bwd(y, ctx, cache, h, recipe)
            add(f"gated, {recipe}, {n} tokens: y, dx, dw", y, dx, dw)
            add(f"norm of {n}, backward", *fp.fp8_rmsnorm_bwd(dx, o["r"], o["rstd"], ones))
    clip = fp.GradClip([g.clone() for g in GRADS])
    norm, out = clip.clip(1.0)
    add("clipping", norm, *out)
    for kw in (dict(score="sigmoid", bias=BIAS, groups=8, groups_kept=3, group_top=2), dict(score="softmax", renormalize=False)):
        w, e = fp.fp8_route_fwd(LOGITS, 6, **kw)
        d = fp.fp8_route_bwd(DW, LOGITS, w, e, score=kw["score"], renormalize=kw.get("renormalize", True))
        order = fp.fp8_expert_order(e, 64, align=16)
        xs = fp.fp8_expert_gather(ROWS, order, out=torch.zeros((order.rows, 512), dtype=torch.bfloat16, device=dev))
        y = fp.fp8_expert_combine(xs, order, w)
        dz, dweights = fp.fp8_expert_combine_bwd(DROWS, xs, order, w, dz=torch.zeros_like(xs))
        add(f"routing, {kw['score']}: weights, experts, dlogits", w, e, d)
        add(f"rows, {kw['score']}", order.counts, order.offsets, order.position, xs, y, dz, dweights,
            fp.fp8_expert_combine(dz, order))
    for i, (w, tokens) in enumerate(zip(W4, ((1, 16, 40), (1, 7, 12, 40), (1, 40, 100)))):
        q = fp.fp8_w4_quantize(w, 64, i == 1)
        add(f"4-bit weight {i}", q.codes, q.scale, q.zero)
        for n in tokens:
            x = normal((n, w.shape[1]), 1.0, n)
            add(f"4-bit products, weight {i}, {n} tokens", fp.fp8_w4_linear(x, q), fp.fp8_w4_gated(x, q))
    gu, dn = fp.fp8_w4_quantize(GU), fp.fp8_w4_quantize(DN, 32, True)
    for n in (1, 9, 150):
        w, e = fp.fp8_route_fwd(LOGITS[:n, :8].contiguous(), 2)
        add(f"4-bit experts, {n} tokens", fp.fp8_w4_experts(normal((n, 1024), 1.0, n), w, e, gu, dn))
    torch.cuda.synchronize()


sequence()
first = sums[:]
names.clear(), sums.clear()
sequence()
print(json.dumps({"status": fp.fp8_get_device_status(), "names": names, "first": first, "second": sums}))
'''


def _run(tmp_path, pdl):
    script = tmp_path / "launch_mode_by_name_child.py"
    script.write_text(CHILD)
    env = dict(os.environ, FP8LIN_PDL=pdl, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, str(script)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def _differ(names, a, b):
    return [n for n, x, y in zip(names, a, b, strict=True) if x != y]


@pytest.mark.gpu
def test_every_output_is_the_same_in_both_modes(tmp_path):
    plain, overlapped = _run(tmp_path, "0"), _run(tmp_path, "1")
    assert plain["status"] == 0 and overlapped["status"] == 0
    names = plain["names"]
    assert names == overlapped["names"] and len(names) > 100
    assert not _differ(names, plain["first"], plain["second"]), "plain launches: two passes differ"
    assert not _differ(names, overlapped["first"], overlapped["second"]), "overlapped launches: two passes differ"
    assert not _differ(names, plain["first"], overlapped["first"]), "plain and overlapped launches differ"
