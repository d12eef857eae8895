"""The norm of a very large set of gradients.

With u = 2^-24: a thread closes its four fp32 sums after each chunk of 32768
elements: 16 u, 2 u to join them, the chunks as pairs, then 5 shuffle steps and
16 warps: 40 u, half of it by the root, which adds 1 u.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


def test_norm_of_a_very_large_set(fp):
    """One value 2^31 times: every addition of a long fp32 chain rounds the same
    way, 430 u of the norm at this value."""
    n, c = 1 << 31, 1.0 + 70 / 128
    g = torch.full((n,), c, dtype=torch.bfloat16, device="cuda")
    norm = float(fp.GradClip([g]).norm())
    del g
    torch.cuda.empty_cache()
    want = math.sqrt(n) * c
    assert abs(norm - want) <= 21 * U * want, (norm - want) / want / U
