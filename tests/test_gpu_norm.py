"""RMS norm with the residual's addition and its FP8 output, forward and
backward, against a plain 64-bit statement.

Tolerances, with u = 2^-24 (fp32) and 2^-8 (bf16, 8 significand bits):
  * a sum of squares is formed from at most 32 terms per thread, 5 shuffle
    steps and 16 warps: 53 u; the root halves it, and the mean, eps and root
    round once each: rstd within 30 u.  y = r * rstd * w adds two roundings,
    a scale two more: within 34 u.
  * an FP8 code stands for its value within half a step of the grid there (and
    the value itself is known within 36 u).
  * dx: three fp32 products and two sums, and a row sum of at most 16 + 5 + 32
    terms: 70 u of the sum of the magnitudes added, then one bf16 rounding.
  * dw: the longest chain is the rows of one group, the groups of a CTA and
    the CTAs: that many u of the sum of magnitudes (and 40 u for rstd).
"""
import pytest
import torch

import ref64 as ref

pytestmark = pytest.mark.gpu
U = ref.EPS24


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


def _inputs(R, C, seed, w_dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((R, C), generator=g)
    x[:, :max(1, C // 100)] *= 30.0
    t = dict(x=x, res=torch.randn((R, C), generator=g), dy=torch.randn((R, C), generator=g) * 1e-2,
             dr=torch.randn((R, C), generator=g) * 1e-2)
    t = {k: v.to(torch.bfloat16).cuda() for k, v in t.items()}
    t["w"] = (1 + 0.2 * torch.randn(C, generator=g)).to(w_dtype).cuda()
    return t


def _check_codes(byte, y, scale, what):
    """Codes of y [R, C] (fp64) under scale [R, ceil(C/128)], one per 1x128 block."""
    v = y * scale.double().repeat_interleave(128, 1)[:, : y.shape[1]]
    got = ref.decode(byte, "e4m3")
    e = torch.clamp(torch.frexp(v.abs())[1].double() - 1, min=-6.0)
    half = torch.exp2(e - 4) * (1 + 1e-9)  # half a step; a value at a binade's end may round up into it
    lim = torch.clamp(v, -448.0, 448.0)
    bad = (got - lim).abs() > half + 36 * U * v.abs()
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} codes off"


def _check_scale(scale, inv, y, what):
    s, _ = ref.scale_of(torch.nn.functional.pad(y.abs(), (0, -y.shape[1] % 128)).view(
        y.shape[0], -1, 128).amax(-1), "e4m3")
    assert torch.all((scale.double() - s).abs() <= 34 * U * s), what
    assert torch.equal(inv, 1.0 / scale), what  # fp32, one division


@pytest.mark.parametrize("R,C", [(1, 16), (1, 4096), (2, 128), (17, 144), (127, 272), (128, 256), (129, 512),
                                 (300, 1040), (64, 2064), (33, 4112), (40, 8192), (5, 8208), (3, 16384),
                                 (5003, 144), (9001, 512), (5111, 1040), (1301, 4096), (1217, 8192), (400, 16384)])
@pytest.mark.parametrize("residual", [True, False])
def test_forward(fp, R, C, residual):
    t = _inputs(R, C, R * 7 + C)
    o = fp.fp8_rmsnorm_fwd(t["x"], t["w"], residual=t["res"] if residual else None, eps=1e-5, bf16=True)
    r = (t["x"].float() + t["res"].float()).to(torch.bfloat16) if residual else t["x"]
    assert torch.equal(o["r"], r)
    rd = r.double()
    rstd = (rd.square().mean(1) + 1e-5) ** -0.5
    assert torch.all((o["rstd"].double() - rstd).abs() <= 30 * U * rstd)
    y = rd * rstd[:, None] * t["w"].double()
    assert torch.all((o["y"].double() - y).abs() <= (ref.EPS8 + 34 * U) * y.abs() * (1 + ref.EPS8))
    _check_scale(o["row_scale"], o["row_scale_inv"], y, "row scales")
    _check_codes(o["row"], y, o["row_scale"], "row")
    assert o["col"].shape == (C, -(-R // 16) * 16)
    yt = y.t().contiguous()
    _check_scale(o["col_scale"], o["col_scale_inv"], yt, "col scales")
    _check_codes(o["col"][:, :R].contiguous(), yt, o["col_scale"], "col")
    assert int(o["col"][:, R:].count_nonzero()) == 0
    assert fp.fp8_get_device_status() == 0


@pytest.mark.parametrize("kw", [dict(rowwise=False), dict(colwise=False), dict(rowwise=False, colwise=False, bf16=True)])
@pytest.mark.parametrize("w_dtype", [torch.float32, torch.bfloat16])
def test_single_outputs_equal_the_full_call(fp, kw, w_dtype):
    t = _inputs(200, 768, 5, w_dtype)
    full = fp.fp8_rmsnorm_fwd(t["x"], t["w"], residual=t["res"], bf16=True)
    part = fp.fp8_rmsnorm_fwd(t["x"], t["w"], residual=t["res"], **kw)
    for k, v in part.items():
        if v is not None:
            assert torch.equal(v, full[k]), k


def test_in_place_residual_and_reused_buffers(fp):
    t = _inputs(130, 512, 6)
    a = fp.fp8_rmsnorm_fwd(t["x"], t["w"], residual=t["res"])
    a = {k: v.clone() for k, v in a.items() if v is not None}
    buf = fp.rmsnorm_buffers(130, 512, "cuda")
    buf["r"] = t["res"]
    b = fp.fp8_rmsnorm_fwd(t["x"], t["w"], residual=t["res"], out=buf)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    assert b["r"].data_ptr() == t["res"].data_ptr()


def test_zero_and_nonfinite_rows(fp):
    """An all-zero row gives zeros and unit scales; a row with a NaN or an
    infinity stays inside its own row (its column blocks ignore NaN)."""
    t = _inputs(140, 256, 8)
    x = t["x"]
    x[3] = 0
    x[5, 7] = float("nan")
    x[6, 9] = float("inf")
    o = fp.fp8_rmsnorm_fwd(x, t["w"])
    clean = x.clone()
    clean[5:7] = 0
    c = fp.fp8_rmsnorm_fwd(clean, t["w"])
    assert int(o["row"][3].count_nonzero()) == 0 and torch.all(o["row_scale"][3] == 1)
    assert torch.all(o["row"][5] == 0x7F)  # NaN through rstd
    assert int(o["row"][6, 9]) == 0x7F     # inf * 0
    keep = [i for i in range(140) if i not in (5, 6)]
    assert torch.equal(o["row"][keep], c["row"][keep])
    assert torch.equal(o["col_scale"], c["col_scale"])
    assert torch.equal(o["col"][:, keep], c["col"][:, keep])


@pytest.mark.parametrize("R,C", [(1, 16), (1, 4096), (9, 144), (129, 512), (1500, 528), (2500, 1024), (300, 2064),
                                 (700, 4096), (50, 8192), (3, 16384), (9001, 272), (1999, 4112), (700, 16384)])
@pytest.mark.parametrize("stream_grad", [True, False])
def test_backward(fp, R, C, stream_grad):
    t = _inputs(R, C, R + C)
    dr = t["dr"] if stream_grad else None
    rstd = ((t["x"].double().square().mean(1) + 1e-6) ** -0.5).float()
    dx, dw = fp.fp8_rmsnorm_bwd(t["dy"], t["x"], rstd, t["w"], dr=dr)
    r, s, dy, w = t["x"].double(), rstd.double()[:, None], t["dy"].double(), t["w"].double()
    g = dy * w
    c = (g * r).mean(1, keepdim=True)
    ref_dx = s * g - r * s ** 3 * c + (dr.double() if stream_grad else 0)
    mag = s * g.abs() + r.abs() * s ** 3 * (g * r).abs().mean(1, keepdim=True) + (dr.double().abs() if stream_grad else 0)
    assert torch.all((dx.double() - ref_dx).abs() <= ref.EPS8 * ref_dx.abs() + 72 * U * mag)
    xh = dy * r * s
    ctas = fp.rmsnorm_workspace(R, C, "cuda").numel() // (4 * C)
    chain = -(-R // ctas) + ctas + 8 + 40
    assert torch.all((dw.double() - xh.sum(0)).abs() <= chain * U * xh.abs().sum(0))
    again = fp.fp8_rmsnorm_bwd(t["dy"], t["x"], rstd, t["w"], dr=dr)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    # in place of either gradient
    buf = t["dy"].clone()
    assert torch.equal(fp.fp8_rmsnorm_bwd(buf, t["x"], rstd, t["w"], dr=dr, dx=buf)[0], dx)


def test_backward_against_differences(fp):
    """Directional derivative of sum(dy * y) + sum(dr * r): central differences
    in 64 bits (step 1e-4: the cubic term is below 1e-6 of the terms added)
    against the kernel's dx (bf16: 2^-8 per element) and dw (fp32)."""
    R, C = 37, 272
    t = _inputs(R, C, 11)
    x, w, dy, dr = (t[k].double() for k in ("x", "w", "dy", "dr"))

    def loss(x, w):
        y = x * (x.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * w
        return (dy * y).sum() + (dr * x).sum()

    rstd = ((x.square().mean(1) + 1e-6) ** -0.5).float()
    dx, dw = fp.fp8_rmsnorm_bwd(t["dy"], t["x"], rstd, t["w"], dr=t["dr"])
    g = torch.Generator().manual_seed(1)
    vx = torch.randn((R, C), generator=g).double().cuda()
    vw = torch.randn(C, generator=g).double().cuda()
    h = 1e-4
    d = float((loss(x + h * vx, w) - loss(x - h * vx, w)) / (2 * h))
    terms = (dx.double() * vx)
    assert abs(float(terms.sum()) - d) <= (2 * ref.EPS8 + 1e-6) * float(terms.abs().sum())
    d = float((loss(x, w + h * vw) - loss(x, w - h * vw)) / (2 * h))
    terms = dw.double() * vw
    assert abs(float(terms.sum()) - d) <= 1e-4 * float(terms.abs().sum())


def test_no_rows(fp):
    w = torch.ones(256, device="cuda")
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    o = fp.fp8_rmsnorm_fwd(e, w)
    assert o["row"].shape == (0, 256)
    dx, dw = fp.fp8_rmsnorm_bwd(e, e, torch.empty(0, device="cuda"), w)
    assert int(dw.count_nonzero()) == 0


def test_side_stream(fp):
    """Inputs made on one stream, the norm run on another that waits for it."""
    t = _inputs(256, 1024, 12)
    want = fp.fp8_rmsnorm_fwd(t["x"], t["w"], residual=t["res"])
    s = torch.cuda.Stream()
    x = t["x"].clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fp.fp8_rmsnorm_fwd(x, t["w"], residual=t["res"])
        dx, dw = fp.fp8_rmsnorm_bwd(t["dy"], got["r"], got["rstd"], t["w"])
    s.synchronize()
    for k in ("r", "row", "col", "row_scale_inv", "col_scale_inv"):
        assert torch.equal(got[k], want[k]), k
    a, b = fp.fp8_rmsnorm_bwd(t["dy"], want["r"], want["rstd"], t["w"])
    assert torch.equal(a, dx) and torch.equal(b, dw)


def test_refusals(fp):
    t = _inputs(32, 256, 13)
    x, w = t["x"], t["w"]
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_fwd(x.float(), w)
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_fwd(x[:, ::2], w)
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_fwd(x, w[:128])
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_fwd(x, w.half())
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_fwd(x, w, residual=t["res"][:16])
    with pytest.raises(fp.FP8Error):
        fp.fp8_rmsnorm_fwd(x, w, eps=0.0)
    with pytest.raises(fp.FP8Error):
        fp.fp8_rmsnorm_fwd(x[:, :100].contiguous(), w[:100].contiguous())
    with pytest.raises(ValueError):
        fp.fp8_rmsnorm_bwd(t["dy"], x, torch.ones(31, device="cuda"), w)
