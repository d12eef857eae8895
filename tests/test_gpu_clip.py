"""Global gradient norm and clipping against a plain 64-bit statement.

Tolerances, with u = 2^-24: a thread adds at most 4096 squares in a row into
four sums (a chain of 1100 at most here), then 5 shuffle steps, 16 warps and
a sum of fp32 pairs; the root halves the relative error: norm within 600 u.  coef adds
three roundings, a product one, and a bf16 result its own 2^-8 (8 significand bits).
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


def _grads(sizes, dtypes, sigma=1e-2, seed=0):
    g = torch.Generator().manual_seed(seed + sum(sizes))
    return [(torch.randn(n, generator=g) * sigma).to(d).cuda()
            for n, d in zip(sizes, dtypes * (len(sizes) // len(dtypes) + 1))]


def _check(norm, out, grads, max_norm):
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(norm) - want) <= 600 * U * want
    coef = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(grads, out):
        e = g.double() * coef
        tol = (2.0 ** -8 if g.dtype == torch.bfloat16 else 0.0) + 610 * U
        assert torch.all((o.double() - e).abs() <= tol * e.abs() * 1.01 + 1e-45)


@pytest.mark.parametrize("sizes", [[1], [7], [2047, 2048, 2049], [515] * 9, [100000, 3, 0, 65536, 1], [5_000_011],
                                   [1 << 20] * 5 + [33]])
@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], [torch.float32, torch.bfloat16]])
@pytest.mark.parametrize("max_norm", [0.01, 1e6])
def test_clip(fp, sizes, dtypes, max_norm):
    grads = _grads(sizes, dtypes)
    out = [torch.full_like(g, 7) for g in grads]
    norm, got = fp.GradClip(grads, out).clip(max_norm)
    _check(norm, got, grads, max_norm)
    if max_norm > 1:  # no clipping: bit for bit
        for g, o in zip(grads, out):
            assert torch.equal(g, o)
    # the same plan again, and in place
    again = fp.GradClip(grads, [torch.empty_like(g) for g in grads])
    n2, o2 = again.clip(max_norm)
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(got, o2))
    inplace = [g.clone() for g in grads]
    n3, o3 = fp.GradClip(inplace).clip(max_norm)
    assert torch.equal(norm, n3) and all(torch.equal(a, b) for a, b in zip(got, o3))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unaligned_views(fp, dtype):
    """Tensors that start off a 16-byte boundary take the element path; their
    neighbours stay untouched."""
    base = _grads([10007], [dtype])[0]
    src = base[3:9000]
    buf = torch.zeros(10007, dtype=dtype, device="cuda")
    norm, got = fp.GradClip([src], [buf[5:9002]]).clip(0.01)
    _check(norm, got, [src], 0.01)
    assert int(buf[:5].count_nonzero()) == 0 and int(buf[9002:].count_nonzero()) == 0


def test_norm_alone_writes_nothing_else(fp):
    grads = _grads([4097, 100], [torch.float32])
    keep = [g.clone() for g in grads]
    c = fp.GradClip(grads)
    n = c.norm().clone()
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    assert torch.equal(n, c.clip(1e30)[0])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_nonfinite_norm_leaves_gradients(fp, bad):
    grads = _grads([5000, 300], [torch.float32, torch.bfloat16])
    grads[0][4321] = bad
    keep = [g.clone() for g in grads]
    norm, out = fp.GradClip(grads).clip(0.5)
    assert not math.isfinite(float(norm))
    for a, b in zip(out, keep):
        assert torch.equal(a.nan_to_num(1.0), b.nan_to_num(1.0))


def test_zero_and_no_gradients(fp):
    z = [torch.zeros(1000, device="cuda")]
    norm, out = fp.GradClip(z).clip(1.0)
    assert float(norm) == 0.0 and int(out[0].count_nonzero()) == 0
    assert float(fp.GradClip([]).clip(1.0)[0]) == 0.0


def test_refusals(fp):
    g = _grads([100], [torch.float32])
    with pytest.raises(ValueError):
        fp.GradClip([g[0].half()])
    with pytest.raises(ValueError):
        fp.GradClip(g, [])
    with pytest.raises(ValueError):
        fp.GradClip([g[0].view(10, 10).t()])
    with pytest.raises(ValueError):
        fp.GradClip(g, [g[0].bfloat16()])
    c = fp.GradClip(g)
    for bad in (0.0, -1.0, float("nan")):
        with pytest.raises(fp.FP8Error):
            c.clip(bad)


@pytest.mark.parametrize("n", [100, 200_000])
@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 1e30])
def test_nonfinite_norm_keeps_its_kind(fp, n, bad):
    """One kernel for small sets, two for larger ones: an infinite sum (1e30
    squared among them) gives an infinite norm, a NaN gives a NaN."""
    grads = _grads([n, 33], [torch.float32])
    grads[0][n // 2] = bad
    norm, out = fp.GradClip(grads, [torch.empty_like(g) for g in grads]).clip(0.5)
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    for a, b in zip(out, grads):
        assert torch.equal(a.nan_to_num(1.0), b.nan_to_num(1.0))


@pytest.mark.parametrize("count", [1, 15, 16, 17, 40])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_sets_at_any_alignment(fp, count, dtype):
    base = _grads([count * 2100], [dtype])[0]
    src = [base[i * 2100 + i % 9:][:1 + (i * 293) % 2048] for i in range(count)]
    buf = torch.zeros(count * 2100, dtype=dtype, device="cuda")
    out = [buf[i * 2100 + i % 9:][:s.numel()] for i, s in enumerate(src)]
    norm, got = fp.GradClip(src, out).clip(0.01)
    _check(norm, got, src, 0.01)
    keep = buf.clone()
    for o in out:
        o.zero_()
    assert int(buf.count_nonzero()) == 0 and int(keep.count_nonzero()) > 0  # nothing written beside them
