"""4-bit products at the ends of their range: one token with more slots than experts, and prompts."""
import pytest
import torch

from test_gpu_w4 import UB, fp, gated, product, weight  # noqa: F401  (the library, loaded once)

pytestmark = pytest.mark.gpu


def experts(x, e, w, vgu, vdn, act):
    """fp8_w4_experts in 64 bits and its bound before the last rounding, on the GPU."""
    k = e.shape[1]
    want = torch.zeros((x.shape[0], vdn.shape[1]), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    for i in range(vgu.shape[0]):
        t, j = (e == i).nonzero(as_tuple=True)
        if t.numel():
            h, eh = gated(x.double()[t], vgu[i].cuda(), act)
            eh = eh * 1.01 + h.abs() * UB * 1.01
            z, ez = product(h, vdn[i].cuda())
            ez = ez * (1 + UB) + eh @ vdn[i].cuda().abs().t()
            ww = w.double()[t, j][:, None]
            want.index_add_(0, t, ww * z)
            bound.index_add_(0, t, ww.abs() * (ez + z.abs() * (k + 2) * 2.0 ** -24))
    return want, bound


@pytest.mark.parametrize("E,k,K,F,N", [
    (1, 17, 2048, 2048, 2048), (2, 64, 2048, 2048, 1040), (1, 17, 256, 16384, 512), (1, 40, 32, 16384, 512),  # tcgen05
    (2, 48, 2048, 2048, 1040),
    (2, 60, 4096, 1024, 64), (1, 2, 512, 256, 512), (3, 4, 96, 64, 48), (4, 300, 256, 96, 64), (1, 70000, 32, 32, 16)])
@pytest.mark.parametrize("group,zero,act", [(32, True, "silu"), (128, False, "gelu")])
@pytest.mark.parametrize("kind", ["random", "one", "holes", "none"])
def test_one_token_with_more_slots_than_experts(fp, E, k, K, F, N, group, zero, act, kind):  # noqa: F811
    gu, vgu = weight(fp, (E, 2 * F, K), group, zero, E + k)
    dn, vdn = weight(fp, (E, N, F), group, zero, E + F)
    g = torch.Generator().manual_seed(k)
    x = torch.randn((1, K), generator=g).bfloat16().cuda()
    e = torch.randint(0, E, (1, k), generator=g, dtype=torch.int32)
    w = torch.rand((1, k), generator=g).cuda()
    if kind == "one":
        e[:] = E - 1
    elif kind == "holes":
        e[torch.rand((1, k), generator=g) < 0.5] = -1
        e[0, k - 1] = E + 3
    elif kind == "none":
        e[:] = -1
    e = e.cuda()
    ws = fp.w4_experts_workspace(1, k, gu, dn).fill_(0xff)  # whatever is read before it is written shows
    out = torch.full((2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = fp.fp8_w4_experts(x, w, e, gu, dn, act, ws=ws, out=out[:1])
    want, bound = experts(x, e, w, vgu, vdn, act)
    assert bool(((y.double() - want).abs() <= bound + want.abs() * UB + 1e-38).all())
    assert bool((out[1] == 7.0).all())
    assert torch.equal(fp.fp8_w4_experts(x, w, e, gu, dn, act), y) and fp.fp8_get_device_status() == 0


@pytest.mark.parametrize("N,K", [(2064, 4128), (2048, 544)])
@pytest.mark.parametrize("T", [1000, 4099])
def test_prompt(fp, N, K, T):  # noqa: F811
    w, v = weight(fp, (N, K), 64, True, N)
    v = v.cuda()
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
    out = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = fp.fp8_w4_linear(x, w, out=out[:T]).double()
    want, bound = product(x.double(), v)
    assert bool(((y - want).abs() <= bound + want.abs() * UB + 1e-38).all()) and bool((out[T] == 7.0).all())
    if N % 32 == 0:
        h = fp.fp8_w4_gated(x, w, "silu").double()
        want, bound = gated(x.double(), v, "silu")
        assert bool(((h - want).abs() <= (bound + want.abs() * UB) * 1.01 + 1e-38).all())


@pytest.mark.parametrize("T,E,k,K,F,N", [(2500, 4, 2, 544, 1024, 1040), (3001, 16, 3, 128, 64, 64), (700, 5, 3, 1056, 1024, 1040),
                                         (4000, 200, 2, 256, 96, 160), (16500, 1000, 2, 256, 256, 32)])
def test_prompt_of_experts(fp, T, E, k, K, F, N):  # noqa: F811
    gu, vgu = weight(fp, (E, 2 * F, K), 64, True, 1)
    dn, vdn = weight(fp, (E, N, F), 64, False, 2)
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, K), generator=g).bfloat16().cuda()
    e = torch.randint(0, max(1, 3 * E // 4), (T, k), generator=g, dtype=torch.int32)  # the last quarter without a token
    e[: T // 3] = 1                                   # one long list, the same expert in each slot
    e[T // 3:][e[T // 3:] % 5 == 2] = 0               # others without one between them
    e[torch.rand((T, k), generator=g) < 0.1] = -1
    e, w = e.cuda(), torch.rand((T, k), generator=g).cuda()
    y = fp.fp8_w4_experts(x, w, e, gu, dn)
    want, bound = experts(x, e, w, vgu, vdn, "silu")
    assert bool(((y.double() - want).abs() <= bound + want.abs() * UB + 1e-38).all())
