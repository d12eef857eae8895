"""CPU-side checks of the routing, row and 4-bit calls: every refusal answers
before anything is launched."""
import ctypes

import pytest

P = ctypes.c_void_p
OK, ARG, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 7, 8
A, ODD8, ODD2, ODD1 = P(1 << 20), P((1 << 20) + 8), P((1 << 20) + 2), P((1 << 20) + 1)   # never dereferenced


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


@pytest.fixture(scope="module")
def L(fp):
    return fp.lib()


def _call(L, f, a, kw, want):
    a = {**a, **kw}
    n = L.fp8_launch_count()
    assert f(*a.values()) == want
    assert L.fp8_launch_count() == n


ROUTE = dict(l=A, dt=1, bias=None, T=5, E=64, k=8, score=0, groups=1, kept=1, top=1, renorm=1, scale=1.0, w=A, e=A,
             st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ARG), (dict(E=0), ARG), (dict(k=0), ARG), (dict(k=65), ARG), (dict(dt=2), ARG), (dict(score=2), ARG),
    (dict(groups=0), ARG), (dict(groups=5), ARG), (dict(groups=8, kept=9), ARG), (dict(groups=8, kept=0), ARG),
    (dict(groups=8, kept=1, k=9), ARG), (dict(top=0), ARG), (dict(top=3), ARG), (dict(scale=0.0), ARG),
    (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(E=1025), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(groups=64, kept=64), UNSUPPORTED),
    (dict(T=1 << 31), SHAPE), (dict(l=None), ARG), (dict(w=None), ARG), (dict(e=None), ARG), (dict(l=ODD2), ALIGN),
    (dict(l=ODD1, dt=0), ALIGN), (dict(T=0, l=None), OK)])
def test_route_forward(L, kw, want):
    _call(L, L.fp8_route_fwd, ROUTE, kw, want)


@pytest.mark.parametrize("kw,want", [
    (dict(dw=None), ARG), (dict(l=None), ARG), (dict(w=None), ARG), (dict(e=None), ARG), (dict(d=None), ARG),
    (dict(d=ODD2), ALIGN), (dict(l=ODD1, dt=0), ALIGN), (dict(k=65), ARG), (dict(E=2048), UNSUPPORTED),
    (dict(scale=0.0), ARG), (dict(score=-1), ARG), (dict(T=0, d=None), OK)])
def test_route_backward(L, kw, want):
    a = dict(dw=A, l=A, dt=1, w=A, e=A, T=5, E=64, k=8, score=0, renorm=1, scale=1.0, d=A, st=None)
    _call(L, L.fp8_route_bwd, a, kw, want)


def test_rows_of_an_order(L):
    rows = L.fp8_expert_rows
    assert rows(10, 4, 1) == 10 and rows(0, 4, 16) == 0 and rows(1, 1024, 16) == 16
    assert rows(37, 3, 16) == 96      # at most 3 gaps of 15, in sixteens
    # whatever the choice: worst case over every split of 9 slots between 3 experts
    worst = max(sum(-(-n // 5) * 5 for n in (a, b, 9 - a - b)) for a in range(10) for b in range(10 - a))
    assert rows(9, 3, 5) >= worst
    b = ctypes.c_size_t()
    size = L.fp8_expert_order_workspace_size
    assert size(2048, 7, ctypes.byref(b)) == OK and b.value == 0
    assert size(2049, 7, ctypes.byref(b)) == OK and b.value == 2 * 7 * 4
    assert size(5, 1025, ctypes.byref(b)) == UNSUPPORTED and size(-1, 4, ctypes.byref(b)) == ARG
    assert size(5, 4, None) == ARG


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), ARG), (dict(E=0), ARG), (dict(align=0), ARG), (dict(align=1025), SHAPE), (dict(E=1025), UNSUPPORTED),
    (dict(counts=None), ARG), (dict(offsets=None), ARG), (dict(position=None), ARG), (dict(order=None), ARG),
    (dict(e=None), ARG), (dict(n=5000, ws=None), WORKSPACE), (dict(n=5000, size=16), WORKSPACE), (dict(n=1 << 31), SHAPE)])
def test_order(L, kw, want):
    a = dict(e=A, n=64, E=8, align=16, counts=A, offsets=A, position=A, order=A, ws=A, size=1 << 30, st=None)
    _call(L, L.fp8_expert_order, a, kw, want)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ARG), (dict(C=8), SHAPE), (dict(C=(1 << 20) + 16), SHAPE), (dict(k=0), ARG), (dict(E=1025), UNSUPPORTED),
    (dict(align=0), ARG), (dict(x=None), ARG), (dict(counts=None), ARG), (dict(offsets=None), ARG),
    (dict(position=None), ARG), (dict(xs=None), ARG), (dict(x=ODD8), ALIGN), (dict(xs=ODD8), ALIGN), (dict(T=0), OK),
    (dict(C=0), OK), (dict(T=1 << 31), SHAPE)])
def test_gather(L, kw, want):
    a = dict(x=A, T=5, C=64, k=2, E=8, align=16, counts=A, offsets=A, position=A, xs=A, st=None)
    _call(L, L.fp8_expert_gather, a, kw, want)


@pytest.mark.parametrize("kw,want", [
    (dict(z=None), ARG), (dict(position=None), ARG), (dict(y=None), ARG), (dict(z=ODD8), ALIGN), (dict(y=ODD8), ALIGN),
    (dict(C=40), SHAPE), (dict(k=-1), ARG), (dict(T=0), OK)])
def test_combine(L, kw, want):
    a = dict(z=A, T=5, C=64, k=2, position=A, w=None, y=A, st=None)
    _call(L, L.fp8_expert_combine, a, kw, want)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), ARG), (dict(z=None), ARG), (dict(w=None), ARG), (dict(dz=None), ARG), (dict(dw=None), ARG),
    (dict(counts=None), ARG), (dict(dy=ODD8), ALIGN), (dict(z=ODD8), ALIGN), (dict(dz=ODD8), ALIGN), (dict(C=24), SHAPE),
    (dict(T=0), OK)])
def test_combine_backward(L, kw, want):
    a = dict(dy=A, z=A, T=5, C=64, k=2, E=8, align=16, counts=A, offsets=A, position=A, w=A, dz=A, dw=A, st=None)
    _call(L, L.fp8_expert_combine_bwd, a, kw, want)


def _weight(fp, **kw):
    a = dict(codes=1 << 20, scale=1 << 20, zero=None, E=1, rows=64, K=256, group=128)
    a.update(kw)
    return fp._W4(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=40), SHAPE), (dict(K=48), SHAPE), (dict(group=16), ARG), (dict(E=0), ARG), (dict(E=1025), UNSUPPORTED),
    (dict(E=2), ARG), (dict(codes=None), ARG), (dict(scale=None), ARG), (dict(codes=(1 << 20) + 8), ALIGN),
    (dict(scale=(1 << 20) + 2), ALIGN), (dict(zero=(1 << 20) + 1), ALIGN), (dict(rows=-16), ARG), (dict(rows=0), OK),
    (dict(rows=1 << 27), SHAPE), (dict(K=1 << 27), SHAPE)])
def test_weights(fp, L, kw, want):
    w = _weight(fp, **kw)
    n = L.fp8_launch_count()
    assert L.fp8_w4_linear(A, 3, w, A, None, 0, None) == want
    if want != ARG or "E" not in kw:
        assert L.fp8_w4_gated(A, 3, w, 0, A, None, 0, None) == want
    assert L.fp8_launch_count() == n


def test_products(fp, L):
    w = _weight(fp)
    n = L.fp8_launch_count()
    f = L.fp8_w4_linear
    assert f(None, 3, w, A, None, 0, None) == ARG and f(A, 3, w, None, None, 0, None) == ARG
    assert f(A, 3, None, A, None, 0, None) == ARG and f(A, -1, w, A, None, 0, None) == ARG
    assert f(ODD8, 3, w, A, None, 0, None) == ALIGN and f(A, 3, w, ODD8, None, 0, None) == ALIGN
    assert f(A, (1 << 18) + 1, w, A, None, 0, None) == SHAPE and f(None, 0, w, None, None, 0, None) == OK
    g = L.fp8_w4_gated
    assert g(A, 3, w, 2, A, None, 0, None) == ARG
    assert g(A, 3, _weight(fp, rows=48), 0, A, None, 0, None) == SHAPE      # F would not be a multiple of 16
    # parts of K that a second kernel sums need a workspace
    big = _weight(fp, K=40960)
    b = ctypes.c_size_t()
    assert L.fp8_w4_workspace_size(big, 20, 0, ctypes.byref(b)) == OK and b.value > 0
    assert f(A, 20, big, A, None, 0, None) == WORKSPACE and f(A, 20, big, A, A, b.value - 1, None) == WORKSPACE
    assert f(A, 20, big, A, ODD8, b.value, None) == ALIGN
    assert L.fp8_w4_workspace_size(w, 3, 0, None) == ARG and L.fp8_w4_workspace_size(None, 3, 0, ctypes.byref(b)) == ARG
    assert L.fp8_w4_workspace_size(w, 3, 1, ctypes.byref(b)) == OK and b.value == 0
    assert L.fp8_launch_count() == n


def test_quantize(L):
    n = L.fp8_launch_count()
    f = L.fp8_w4_quantize
    assert f(None, 16, 32, 32, A, A, A, None) == ARG and f(A, 16, 32, 32, None, A, A, None) == ARG
    assert f(A, 16, 32, 32, A, None, A, None) == ARG and f(A, 16, 32, 48, A, A, A, None) == ARG
    assert f(A, 8, 32, 32, A, A, A, None) == SHAPE and f(A, 16, 40, 32, A, A, A, None) == SHAPE
    assert f(ODD8, 16, 32, 32, A, A, A, None) == ALIGN and f(A, 16, 32, 32, A, ODD8, A, None) == ALIGN
    assert f(None, 0, 32, 32, None, None, None, None) == OK
    assert L.fp8_launch_count() == n


def test_experts(fp, L):
    gu, dn = _weight(fp, E=4, rows=128, K=256), _weight(fp, E=4, rows=96, K=64)
    b = ctypes.c_size_t()
    size = L.fp8_w4_experts_workspace_size
    assert size(3, 2, 4, 256, 64, 96, ctypes.byref(b)) == OK and b.value > 0
    need = b.value
    assert size(3, 2, 4, 256, 64, 96, None) == ARG and size(-1, 2, 4, 256, 64, 96, ctypes.byref(b)) == ARG
    assert size(3, 2, 4, 256, 48, 96, ctypes.byref(b)) == SHAPE and size(3, 2, 2000, 256, 64, 96, ctypes.byref(b)) == UNSUPPORTED
    assert size(0, 2, 4, 256, 64, 96, ctypes.byref(b)) == OK and b.value == 0
    n = L.fp8_launch_count()

    def call(x=A, T=3, k=2, w=A, e=A, gu=gu, dn=dn, act=0, y=A, ws=A, size=need):
        return L.fp8_w4_experts(x, T, k, w, e, gu, dn, act, y, ws, size, None)
    assert call(x=None) == ARG and call(w=None) == ARG and call(e=None) == ARG and call(y=None) == ARG
    assert call(gu=None) == ARG and call(dn=None) == ARG and call(k=0) == ARG and call(T=-1) == ARG and call(act=5) == ARG
    assert call(x=ODD8) == ALIGN and call(y=ODD8) == ALIGN and call(ws=ODD8) == ALIGN
    assert call(ws=None) == WORKSPACE and call(size=need - 1) == WORKSPACE
    assert call(dn=_weight(fp, E=3, rows=96, K=64)) == SHAPE          # another number of experts
    assert call(dn=_weight(fp, E=4, rows=96, K=96)) == SHAPE          # another F
    assert call(T=0, x=None, ws=None) == OK
    assert L.fp8_launch_count() == n


def test_alignment_of_small_arrays(fp, L):
    """Float and int arrays need their type's alignment, no more (4 is fine)."""
    n = L.fp8_launch_count()
    for name in ("w", "e", "bias"):
        assert L.fp8_route_fwd(*{**ROUTE, name: ODD2}.values()) == ALIGN
    for i in (0, 3, 4):
        a = [A, A, 1, A, A, 5, 64, 8, 0, 1, 1.0, A, None]
        a[i] = ODD2
        assert L.fp8_route_bwd(*a) == ALIGN
    for i in (0, 4, 5, 6, 7, 8):
        a = [A, 64, 8, 16, A, A, A, A, A, 1 << 30, None]
        a[i] = ODD2
        assert L.fp8_expert_order(*a) == ALIGN
    for i in (6, 7, 8):
        a = [A, 5, 64, 2, 8, 16, A, A, A, A, None]
        a[i] = ODD2
        assert L.fp8_expert_gather(*a) == ALIGN
    for i in (4, 5):
        a = [A, 5, 64, 2, A, A, A, None]
        a[i] = ODD2
        assert L.fp8_expert_combine(*a) == ALIGN
    for i in (7, 8, 9, 10, 12):
        a = [A, A, 5, 64, 2, 8, 16, A, A, A, A, A, A, None]
        a[i] = ODD2
        assert L.fp8_expert_combine_bwd(*a) == ALIGN
    gu, dn = _weight(fp, E=4, rows=128, K=256), _weight(fp, E=4, rows=96, K=64)
    for i in (3, 4):
        a = [A, 3, 2, A, A, gu, dn, 0, A, A, 1 << 30, None]
        a[i] = ODD2
        assert L.fp8_w4_experts(*a) == ALIGN
    assert L.fp8_launch_count() == n
