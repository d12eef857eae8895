"""The routing, row and 4-bit calls of the binding, run on the host: what they
refuse, what they allocate where, and what they pass on."""
import pytest
import torch

import hostcalls
from hostcalls import FakeStream, Host, bf16, dev, f32

NEW = ("fp8_route_fwd", "fp8_route_bwd", "fp8_expert_order", "fp8_expert_gather", "fp8_expert_combine",
       "fp8_expert_combine_bwd", "fp8_w4_quantize", "fp8_w4_linear", "fp8_w4_gated", "fp8_w4_experts")


@pytest.fixture()
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


@pytest.fixture()
def host(fp, monkeypatch):
    monkeypatch.setattr(hostcalls, "LAUNCHING", hostcalls.LAUNCHING + NEW)
    return Host(fp, monkeypatch)


def i32(*shape):
    return dev(torch.zeros(shape, dtype=torch.int32))


def w4(fp, *shape, group=64, zero=False):
    nb = -(-shape[-1] // group)
    codes = dev(torch.zeros((*shape[:-1], shape[-1] // 2), dtype=torch.uint8))
    z = dev(torch.zeros((*shape[:-1], nb), dtype=torch.uint8)) if zero else None
    return fp.W4Weight(codes, bf16(*shape[:-1], nb), z, group)


def test_route_arguments(fp, host):
    l = f32(5, 64)
    w, e = fp.fp8_route_fwd(l, 8, "sigmoid", bias=f32(64), groups=8, groups_kept=3, group_top=2, renormalize=False, scale=2.5)
    (a,) = host.launches("fp8_route_fwd")
    assert a[:12] == (l.data_ptr(), 1, a[2], 5, 64, 8, 1, 8, 3, 2, False, 2.5) and a[2]
    assert w.shape == e.shape == (5, 8) and w.dtype == torch.float32 and e.dtype == torch.int32
    fp.fp8_route_fwd(bf16(5, 64), 8, groups=4)
    a = host.launches("fp8_route_fwd")[1]
    assert a[1] == 0 and a[2] is None and a[7:9] == (4, 4)        # all groups stay unless told otherwise
    out = fp.fp8_route_fwd(l, 8, out=(w, e))
    assert out[0] is w and out[1] is e
    for bad in (f32(5, 64).t(), dev(torch.zeros((5, 64), dtype=torch.float16)), f32(320)):
        with pytest.raises(ValueError):
            fp.fp8_route_fwd(bad, 8)
    with pytest.raises(ValueError):
        fp.fp8_route_fwd(l, 8, bias=f32(63))
    with pytest.raises(ValueError):
        fp.fp8_route_fwd(l, 8, out=(w, i32(5, 7)))
    with pytest.raises(KeyError):
        fp.fp8_route_fwd(l, 8, "tanh")
    d = fp.fp8_route_bwd(f32(5, 8), l, w, e)
    assert d.shape == l.shape and d.dtype == l.dtype
    for args in ((f32(5, 7), l, w, e), (f32(5, 8), f32(4, 64), w, e), (f32(5, 8), l, f32(5, 9), e)):
        with pytest.raises(ValueError):
            fp.fp8_route_bwd(*args)
    with pytest.raises(ValueError):
        fp.fp8_route_bwd(f32(5, 8), l, w, e, out=bf16(5, 64))


def test_order_and_rows(fp, host):
    e = i32(6, 2)
    o = fp.fp8_expert_order(e, 3, align=16)
    assert o.rows == fp.expert_rows(6, 2, 3, 16) == 64
    assert o.counts.shape == (3,) and o.offsets.shape == (4,) and o.position.shape == (6, 2) and o.order.shape == (64,)
    a = host.launches("fp8_expert_order")[0]
    assert a[4:8] == tuple(t.data_ptr() for t in (o.counts, o.offsets, o.position, o.order)) and a[8] is None
    assert fp.fp8_expert_order(e, 3, align=16, out=o) is o
    for kw in (dict(n_experts=4, align=16), dict(n_experts=3, align=1)):
        with pytest.raises(ValueError):
            fp.fp8_expert_order(e, out=o, **kw)
    for bad in (e.t(), dev(torch.zeros((6, 2), dtype=torch.int64)), i32(12)):
        with pytest.raises(ValueError):
            fp.fp8_expert_order(bad, 3)
    fp.fp8_expert_order(i32(3000, 2), 3)
    assert host.launches("fp8_expert_order")[-1][9] >= 3 * 3 * 4     # many slots: a workspace
    x, z = bf16(6, 32), bf16(64, 32)
    assert fp.fp8_expert_gather(x, o).shape == (64, 32)
    assert fp.fp8_expert_combine(z, o, f32(6, 2)).shape == (6, 32)
    dz, dw = fp.fp8_expert_combine_bwd(x, z, o, f32(6, 2))
    assert dz.shape == z.shape and dw.shape == (6, 2)
    for call in (lambda: fp.fp8_expert_gather(bf16(5, 32), o), lambda: fp.fp8_expert_gather(x, o, out=bf16(63, 32)),
                 lambda: fp.fp8_expert_combine(bf16(63, 32), o), lambda: fp.fp8_expert_combine(z, o, f32(2, 6)),
                 lambda: fp.fp8_expert_combine(z, o, out=bf16(6, 16)),
                 lambda: fp.fp8_expert_combine_bwd(x, bf16(64, 16), o, f32(6, 2)),
                 lambda: fp.fp8_expert_combine_bwd(x, z, o, None),
                 lambda: fp.fp8_expert_combine_bwd(x, z, o, f32(6, 2), dz=bf16(6, 32)),
                 lambda: fp.fp8_expert_gather(dev(torch.zeros((6, 32), dtype=torch.bfloat16), 1), o)):
        with pytest.raises((ValueError, AttributeError)):
            call()


def test_weights(fp, host):
    w = w4(fp, 32, 96, group=32)
    assert (w.E, w.N, w.K, w.stack) == (1, 32, 96, False)
    assert w4(fp, 3, 32, 96, group=128, zero=True).E == 3
    u8, s = dev(torch.zeros((32, 48), dtype=torch.uint8)), bf16(32, 3)
    for args in ((u8, bf16(32, 2), None, 32), (u8, f32(32, 3), None, 32), (u8, s, None, 16),
                 (u8, s, dev(torch.zeros((32, 2), dtype=torch.uint8)), 32), (u8.t(), s, None, 32),
                 (dev(torch.zeros((24, 48), dtype=torch.uint8)), bf16(24, 3), None, 32),
                 (dev(torch.zeros((32, 24), dtype=torch.uint8)), bf16(32, 2), None, 32),
                 (torch.zeros((32, 48), dtype=torch.uint8), s, None, 32), (u8, dev(torch.zeros((32, 3), dtype=torch.bfloat16), 1), None, 32)):
        with pytest.raises(ValueError):
            fp.W4Weight(*args)
    q = fp.fp8_w4_quantize(bf16(2, 16, 64), 32, zero=True)
    assert q.codes.shape == (2, 16, 32) and q.scale.shape == q.zero.shape == (2, 16, 2) and q.stack
    for shape, group in (((16, 48), 32), ((8, 64), 32), ((16, 64), 48), ((64,), 32)):
        with pytest.raises(ValueError):
            fp.fp8_w4_quantize(bf16(*shape), group)


def test_products(fp, host):
    w = w4(fp, 64, 96, group=32)
    assert fp.fp8_w4_linear(bf16(5, 96), w).shape == (5, 64)
    assert fp.fp8_w4_gated(bf16(5, 96), w, "gelu").shape == (5, 32)
    assert host.launches("fp8_w4_linear")[0][4:6] == (None, 0)
    assert host.launches("fp8_w4_gated")[0][3] == 1
    big = w4(fp, 32, 40960)                                        # summed by a second kernel
    fp.fp8_w4_linear(bf16(20, 40960), big)
    a = host.launches("fp8_w4_linear")[1]
    assert a[4] and a[5] == fp.w4_workspace(big, 20).numel()
    for call in (lambda: fp.fp8_w4_linear(bf16(5, 64), w), lambda: fp.fp8_w4_linear(bf16(96), w),
                 lambda: fp.fp8_w4_linear(f32(5, 96), w), lambda: fp.fp8_w4_linear(bf16(96, 5).t(), w),
                 lambda: fp.fp8_w4_linear(bf16(5, 96), w, out=bf16(5, 32)),
                 lambda: fp.fp8_w4_linear(bf16(5, 96), w4(fp, 2, 64, 96, group=32)),
                 lambda: fp.fp8_w4_gated(bf16(5, 96), w4(fp, 48, 96, group=32))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(KeyError):
        fp.fp8_w4_gated(bf16(5, 96), w, "relu")
    with pytest.raises(fp.FP8Error):
        real = fp._w4_bytes(32, 40960, 48, 20, False)              # no such group
        assert real is None


def test_experts(fp, host):
    gu, dn = w4(fp, 4, 128, 96), w4(fp, 4, 96, 64)
    x, w, e = bf16(3, 96), f32(3, 2), i32(3, 2)
    assert fp.fp8_w4_experts(x, w, e, gu, dn).shape == (3, 96)
    a = host.launches("fp8_w4_experts")[0]
    assert a[1:3] == (3, 2) and a[10] == fp.w4_experts_workspace(3, 2, gu, dn).numel()
    for call in (lambda: fp.fp8_w4_experts(bf16(3, 64), w, e, gu, dn), lambda: fp.fp8_w4_experts(x, f32(2, 2), e, gu, dn),
                 lambda: fp.fp8_w4_experts(x, w, i32(4, 2), gu, dn),
                 lambda: fp.fp8_w4_experts(x, w, e, gu, w4(fp, 3, 96, 64)),
                 lambda: fp.fp8_w4_experts(x, w, e, gu, w4(fp, 4, 96, 128)),
                 lambda: fp.fp8_w4_experts(x, w, e, gu, dn, out=bf16(3, 64)),
                 lambda: fp.fp8_w4_experts(x, w, dev(torch.zeros((3, 2), dtype=torch.int64)), gu, dn)):
        with pytest.raises(ValueError):
            call()


def test_another_device_is_refused(fp, host, monkeypatch):
    """The kernels run on the stream's device: tensors of another one are refused before the call."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    w = w4(fp, 64, 96, group=32)
    for call in (lambda: fp.fp8_route_fwd(f32(5, 64), 8), lambda: fp.fp8_expert_order(i32(3, 2), 4),
                 lambda: fp.fp8_w4_linear(bf16(5, 96), w), lambda: fp.fp8_w4_quantize(bf16(16, 64), 32)):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    s = FakeStream(7)
    s.device_index = 0
    fp.fp8_route_fwd(f32(5, 64), 8, stream=s)
    assert host.calls[-1][1][-1] == 7


def test_calls_on_a_stream_allocate_there(fp, host):
    s = FakeStream(77)
    s.device_index = 0
    w = w4(fp, 64, 40960)
    gu, dn = w4(fp, 4, 128, 96), w4(fp, 4, 96, 64)
    host.made.clear()
    ww, e = fp.fp8_route_fwd(f32(3, 4), 2, stream=s)
    fp.fp8_route_bwd(f32(3, 2), f32(3, 4), ww, e, stream=s)
    o = fp.fp8_expert_order(i32(3000, 2), 4, stream=s)
    xs = fp.fp8_expert_gather(bf16(3000, 32), o, stream=s)
    fp.fp8_expert_combine(xs, o, stream=s)
    fp.fp8_expert_combine_bwd(bf16(3000, 32), xs, o, f32(3000, 2), stream=s)
    fp.fp8_w4_quantize(bf16(16, 64), 32, True, stream=s)
    fp.fp8_w4_linear(bf16(20, 40960), w, stream=s)
    fp.fp8_w4_gated(bf16(20, 40960), w, stream=s)
    fp.fp8_w4_experts(bf16(3, 96), f32(3, 2), i32(3, 2), gu, dn, stream=s)
    assert len(host.made) >= 16 and all(at == 77 for _, at in host.made)
    assert [a[-1] for _, a in host.calls] == [77] * len(host.calls) and len(host.calls) == 10
