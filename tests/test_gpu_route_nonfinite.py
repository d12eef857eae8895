"""Gradients of rows whose scores are not numbers: no expert, so nothing passes."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(9, 40, 3), (9, 1000, 8), (6007, 64, 8), (6007, 17, 2)])
def test_rows_without_an_expert_pass_no_gradient(dtype, score, renorm, T, E, k):
    import fp8_mixed_precision_gb300 as fp
    g = torch.Generator().manual_seed(E)
    l = torch.randn((T, E), generator=g).to(dtype)
    l[1, E - 1] = math.nan
    l[2, 3] = math.inf
    l[3, 0], l[3, 5] = math.inf, math.nan
    l[4, 2], l[4, 7] = math.inf, -math.inf
    l[5] = -math.inf
    l[T - 1, 1] = math.inf
    kw = dict(score=score, renormalize=renorm)
    w, e = fp.fp8_route_fwd(l.cuda(), k, **kw)
    dw = torch.randn((T, k), generator=g).cuda()
    d = fp.fp8_route_bwd(dw, l.cuda(), w, e, **kw)
    none = (e == -1).all(1)
    # (an infinite logit has the sigmoid 1)
    assert none.cpu().nonzero().flatten().tolist() == ([1, 2, 3, 4, 5, T - 1] if score == "softmax" else [1, 3, 5])
    assert bool((d[none] == 0).all()) and bool(d.isfinite().all())
    # the other rows are as they are without these
    keep = [0, 6, 7]
    assert torch.equal(d[keep], fp.fp8_route_bwd(dw, l.cuda().nan_to_num(0.0, 0.0, -1.0), w, e, **kw)[keep])
