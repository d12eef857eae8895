"""CPU-side checks of the norm, gated feed-forward and clipping calls: every
refusal answers before anything is launched."""
import ctypes

import pytest

P = ctypes.c_void_p
OK, ARG, SHAPE, ALIGN, STALE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 7, 8
A, ODD = P(1 << 20), P((1 << 20) + 8)   # never dereferenced


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp.lib()


def _norm_args(**kw):
    a = dict(x=A, res=A, w=A, dt=1, rows=5, cols=256, eps=1e-6, r=A, rstd=A, lo=A, y=None, row=A, col=A, rs=A, rsi=A,
             cs=A, csi=A, st=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), ARG), (dict(cols=250), SHAPE), (dict(cols=16400), UNSUPPORTED), (dict(dt=2), ARG),
    (dict(eps=0.0), ARG), (dict(eps=float("nan")), ARG), (dict(row=None, col=None), ARG), (dict(r=None), ARG),
    (dict(res=None), ARG), (dict(rstd=None), ARG), (dict(lo=None), ARG), (dict(rsi=None), ARG), (dict(csi=None), ARG), (dict(w=None), ARG),
    (dict(x=ODD), ALIGN), (dict(w=ODD), ALIGN), (dict(row=ODD), ALIGN), (dict(rows=0), OK)])
def test_norm_forward(L, kw, want):
    n = L.fp8_launch_count()
    assert L.fp8_rmsnorm_fwd(*_norm_args(**kw)) == want
    assert L.fp8_launch_count() == n


def test_norm_backward(L):
    b = ctypes.c_size_t()
    assert L.fp8_rmsnorm_workspace_size(1000, 512, ctypes.byref(b)) == OK and b.value > 0 and b.value % 2048 == 0
    assert L.fp8_rmsnorm_workspace_size(0, 512, ctypes.byref(b)) == OK and b.value == 0
    assert L.fp8_rmsnorm_workspace_size(4, 500, ctypes.byref(b)) == SHAPE

    def call(dy=A, dr=None, r=A, rstd=A, w=A, dt=0, rows=64, cols=256, dx=A, dw=A, ws=A, n=1 << 30):
        return L.fp8_rmsnorm_bwd(dy, dr, r, rstd, w, dt, rows, cols, dx, dw, ws, n, None)

    assert call(dy=None) == ARG and call(dw=None) == ARG and call(rstd=None) == ARG
    assert call(dr=ODD) == ALIGN and call(dw=ODD) == ALIGN
    assert call(n=16) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(cols=40) == SHAPE and call(cols=0) == OK


def test_gated(L):
    b = ctypes.c_size_t()
    assert L.fp8_gated_ctx_size(1, 5, 256, 384, ctypes.byref(b)) == OK
    assert b.value >= 16 * 256 + 4 * 5 * 384
    assert L.fp8_gated_ctx_size(1, 5, 256, 400, ctypes.byref(b)) == SHAPE   # block: whole 128-row tiles
    assert L.fp8_gated_ctx_size(0, 5, 256, 400, ctypes.byref(b)) == OK
    assert L.fp8_gated_ctx_size(0, 5, 250, 400, ctypes.byref(b)) == SHAPE
    assert L.fp8_gated_ctx_size(3, 5, 256, 400, ctypes.byref(b)) == ARG
    s = ctypes.c_size_t()
    assert L.fp8_gated_workspace_size(1, 5, 256, 384, 0, ctypes.byref(s)) == OK
    t = ctypes.c_size_t()
    assert L.fp8_gated_workspace_size(1, 5, 256, 384, 1, ctypes.byref(t)) == OK and t.value >= s.value
    c = P()
    assert L.fp8_weight_cache_create(ctypes.byref(c)) == OK
    h, odd = ctypes.c_int32(), ctypes.c_int32()
    reg = L.fp8_weight_cache_register
    assert reg(c, A, 768, 256, 1, A, A, A, A, A, A, None, 0, ctypes.byref(h)) == OK
    assert reg(c, A, 320, 256, 1, A, A, A, A, A, A, None, 0, ctypes.byref(odd)) == OK
    n = L.fp8_launch_count()
    fwd = L.fp8_gated_fwd
    big = 1 << 40
    assert fwd(A, 5, 256, c, h, 1, 0, A, A, A, big, None) == STALE
    assert fwd(A, 5, 256, c, h, 0, 0, A, A, A, big, None) == ARG       # another recipe
    assert fwd(A, 5, 256, c, h, 1, 2, A, A, A, big, None) == ARG       # no such activation
    assert fwd(A, -1, 256, c, h, 1, 0, A, A, A, big, None) == ARG
    assert fwd(A, 5, 256, c, 7, 1, 0, A, A, A, big, None) == ARG
    assert fwd(A, 5, 256, None, h, 1, 0, A, A, A, big, None) == ARG
    assert fwd(A, 5, 256, c, odd, 1, 0, A, A, A, big, None) == SHAPE
    assert L.fp8_gated_bwd(A, 5, 384, A, c, h, 1, 0, A, A, A, big, None) == STALE
    assert L.fp8_gated_fwd_quantized(A, A, 5, 256, c, h, 1, 0, A, None, None) == STALE
    assert L.fp8_launch_count() == n
    L.fp8_weight_cache_destroy(c)


def test_clip(L):
    from fp8_mixed_precision_gb300 import _GradDesc
    p = P()

    def make(*d):
        return L.fp8_grad_clip_create((_GradDesc * len(d))(*d), len(d), ctypes.byref(p))

    at = 1 << 20
    assert make(_GradDesc(at, at, -1, 1)) == ARG
    assert make(_GradDesc(at, at, 4, 5)) == ARG
    assert make(_GradDesc(None, at, 4, 1)) == ARG
    assert make(_GradDesc(at + 2, at, 4, 1)) == ALIGN
    assert L.fp8_grad_clip_create(None, 1, ctypes.byref(p)) == ARG
    assert make(_GradDesc(at + 2, at, 40_000_000, 0), _GradDesc(None, None, 0, 1)) == OK
    b = ctypes.c_size_t()
    assert L.fp8_grad_clip_table_size(p, ctypes.byref(b)) == OK and b.value % 24 == 0 and b.value > 24 * 1000
    host = (ctypes.c_uint8 * b.value)()
    assert L.fp8_grad_clip_table_write(p, host, b.value - 1) == WORKSPACE
    assert L.fp8_grad_clip_table_write(p, host, b.value) == OK
    n = L.fp8_launch_count()
    run = L.fp8_grad_clip_run
    assert run(p, A, 0.0, A, A, 1 << 20, None) == ARG
    assert run(p, None, 1.0, A, A, 1 << 20, None) == ARG
    assert run(p, A, 1.0, None, A, 1 << 20, None) == ARG
    assert run(p, A, 1.0, A, ODD, 1 << 20, None) == ALIGN
    assert run(p, A, 1.0, A, A, 0, None) == WORKSPACE
    assert L.fp8_grad_norm(None, A, A, A, 1 << 20, None) == ARG
    assert L.fp8_launch_count() == n
    L.fp8_grad_clip_destroy(p)
