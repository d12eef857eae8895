"""The norm's bytes against those of the 64-bit norm.

With u = 2^-24: rstd as a pair lies within 2^-36 of the root (sums of up to 32
squares per thread keep their errors in an fp32 sum, 2^-37 of it at worst; the
pairs that join them and the Newton step are below 2^-42).  y is then the other
neighbour of a rounding with probability 2^-36 / 2^-25 = 2^-11 at worst and
2^-14 on average: scales differ in at most one block in 2000.  A code differs
where such a y, or a y under such a scale, lies within an ulp of a tie, one in
2^-24 / 2^-4: below 10^-9 of the elements, so 2 are allowed.
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


@pytest.mark.parametrize("R,C", [(65536, 512), (4096, 4096), (2048, 8192), (16384, 1040), (100000, 16), (30000, 144),
                                 (1000, 16384), (20000, 272)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_bytes_are_those_of_the_exact_norm(fp, R, C, residual):
    g = torch.Generator(device="cuda").manual_seed(R + C + residual)
    x = torch.randn((R, C), generator=g, device="cuda")
    x[:, torch.randint(0, C, (max(1, C // 256),), generator=g, device="cuda")] *= 20.0
    x[R // 2:] *= torch.exp(2 * torch.randn((R - R // 2, C), generator=g, device="cuda"))  # squares far apart
    x = x.to(torch.bfloat16)
    res = torch.randn((R, C), generator=g, device="cuda").to(torch.bfloat16) if residual else None
    w = 1.0 + 0.1 * torch.randn(C, generator=g, device="cuda")
    o = fp.fp8_rmsnorm_fwd(x, w, residual=res, bf16=True)
    r = o["r"].double()
    rstd = (r.square().mean(1) + 1e-6) ** -0.5
    err = ((o["rstd"].double() + o["rstd_lo"].double()) - rstd).abs() / rstd
    assert float(err.max()) <= 2.0 ** -36, math.log2(float(err.max()))
    y = ref.f32(r * rstd[:, None] * w.double())  # what is quantized: the exact norm in fp32
    assert int((o["y"] != y.float().to(torch.bfloat16)).sum()) <= 2
    for name, v in (("row", y), ("col", y.t().contiguous())):
        q, s, _ = ref.blocks(v, "e4m3")
        got = ref.decode(o[name][:, :v.shape[1]].contiguous(), "e4m3")
        off = int((o[f"{name}_scale"].double() != s.view(o[f"{name}_scale"].shape)).sum())
        assert off <= 2 + s.numel() / 2000, (name, off, s.numel())
        assert int((got != q).sum()) <= 2, name
