"""Routing where fp32 holds none of a row's sigmoid scores: fp64 tells them apart."""
import pytest
import torch

from test_gpu_route import check, fp  # noqa: F401  (the library, loaded once)

pytestmark = pytest.mark.gpu


def rows(T, E, dtype, lo, hi, seed):
    return (lo + (hi - lo) * torch.rand((T, E), generator=torch.Generator().manual_seed(seed))).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lo,hi", [(-88.6, -87.0), (-130.0, -86.0), (-600.0, -104.0)])
@pytest.mark.parametrize("E,k,groups,kept,top", [(32, 6, 1, 1, 1), (64, 5, 8, 2, 2), (64, 8, 4, 2, 1), (256, 8, 8, 3, 2),
                                                 (510, 6, 5, 2, 2)])
@pytest.mark.parametrize("T", [7, 5003])  # (many tokens: fewer lanes to each)
def test_scores_below_fp32(fp, dtype, lo, hi, E, k, groups, kept, top, T):  # noqa: F811
    l = rows(min(T, 40), E, dtype, lo, hi, E)
    for bias in (torch.zeros(E), None):
        check(fp, l, k, "sigmoid", bias, groups, kept, top)
        if T > 40:
            many = l[torch.arange(T) % 40].cuda()
            args = dict(score="sigmoid", bias=None if bias is None else bias.cuda(), groups=groups, groups_kept=kept,
                        group_top=top)
            w, e = fp.fp8_route_fwd(many, k, **args)
            w1, e1 = fp.fp8_route_fwd(many[:40].contiguous(), k, **args)
            at = torch.arange(T) % 40
            assert torch.equal(e, e1[at]) and torch.allclose(w, w1[at], rtol=2.0 ** -18, atol=0)


def test_one_score_within_range(fp):  # noqa: F811
    """A score that fp32 holds beside ones that it does not."""
    l = rows(9, 64, torch.float32, -140.0, -95.0, 1)
    l[:, 40] = -20.0
    l[3:, 10] = 2.0
    check(fp, l, 6, "sigmoid", torch.zeros(64), 8, 3, 2)
    check(fp, l, 6, "sigmoid", torch.full((64,), 2.0 ** -130), 1, 1, 1)
