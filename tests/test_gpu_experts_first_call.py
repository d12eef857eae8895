"""A process whose first call of each operator is captured into a graph: what the
library asks for and sets once (shared memory, clusters that fit, the SM count) needs
no call before, and the replayed results are those of plain calls."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
import fp8_mixed_precision_gb300 as fp
g = torch.Generator(device="cuda").manual_seed(1)
def weight(*shape, group=64):
    return fp.W4Weight(torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), dtype=torch.uint8, device="cuda", generator=g),
                       (torch.rand((*shape[:-1], -(-shape[-1] // group)), device="cuda", generator=g) * 0.02).bfloat16(),
                       None, group)
def rows(*shape):
    return torch.randn(shape, device="cuda", generator=g).bfloat16()
one, wide, gu, dn = weight(512, 8192), weight(8192, 2048), weight(8, 512, 256), weight(8, 256, 256)
x1, xw, x = rows(5, 8192), rows(40, 2048), rows(9, 256)
logits = torch.randn((9, 8), device="cuda", generator=g)
ws1, wsw, wse = fp.w4_workspace(one, 5), fp.w4_workspace(wide, 40, True), fp.w4_experts_workspace(9, 2, gu, dn)
def calls():
    w, e = fp.fp8_route_fwd(logits, 2)
    order = fp.fp8_expert_order(e, 8, align=16)
    xs = fp.fp8_expert_gather(x, order)
    y = fp.fp8_expert_combine(xs, order, w)
    dz, dw = fp.fp8_expert_combine_bwd(x, xs, order, w)
    d = fp.fp8_route_bwd(dw, logits, w, e)
    return [w, e, y, dw, d, fp.fp8_w4_linear(x1, one, ws=ws1), fp.fp8_w4_gated(xw, wide, ws=wsw),
            fp.fp8_w4_experts(x, w, e, gu, dn, ws=wse)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    kept = calls()
for _ in range(2):
    logits.normal_(generator=g)
    x.normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(kept, calls()):
        assert torch.equal(a, b)
assert fp.fp8_get_device_status() == 0
print("first calls captured")
"""


def test_first_calls_in_a_graph():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first calls captured" in r.stdout, r.stderr[-2000:]
