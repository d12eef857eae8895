"""Results of the gated MLP stack and of clipping stay what they were when
later calls run."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp():
    from fp8_mixed_precision_gb300 import build
    build.build()
    import fp8_mixed_precision_gb300 as fp
    return fp


def _normal(shape, sigma, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("recipe", ["block", "tensorwise"])
@pytest.mark.parametrize("layers", [0, 1, 3])
def test_microbatches_and_steps(fp, recipe, layers):
    from fp8_mixed_precision_gb300.gated_mlp import FP8GatedMLPStack
    n, d = 128, 256
    m = FP8GatedMLPStack(d, 256, layers, n, recipe, max_norm=0.25)
    xs, dys = [_normal((n, d), 1.0, i) for i in range(3)], [_normal((n, d), 1e-2, 9 + i) for i in range(3)]
    m.cache.begin_cycle()
    m.version += 1
    got = [m.microbatch(x, dy) for x, dy in zip(xs, dys)]
    for x, dy, (y, dx) in zip(xs, dys, got):
        z, dz = m.microbatch(x, dy)
        assert torch.equal(y, z) and torch.equal(dx, dz)
    assert len({t.data_ptr() for p in got for t in p}) == 6
    norms = [m.step([x], [dy])[0] for x, dy in zip(xs, dys)]
    assert len({float(v) for v in norms}) == 3
    for x, dy, v in zip(xs, dys, norms):
        assert float(m.step([x], [dy])[0]) == float(v)


def test_norms_of_one_plan(fp):
    g = [_normal((5000,), 1e-2, 1), _normal((300,), 1e-2, 2).float()]
    c = fp.GradClip(g)
    before = c.norm()
    during, _ = c.clip(0.1)
    after = c.norm()
    assert float(before) == float(during) > 0.11
    assert abs(float(after) - 0.1) < 1e-3  # bf16 gradients: 2^-8 each, in part


def test_a_plan_keeps_the_memory_it_points_to(fp):
    """Its table holds addresses: memory that a gradient is moved away from must
    not become another tensor's."""
    g, o = torch.zeros(3_000_017, device="cuda"), torch.zeros(3_000_017, device="cuda")
    at = {g.data_ptr(), o.data_ptr()}
    plan = fp.GradClip([g], [o])
    g.data, o.data = torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")
    new = [torch.empty(3_000_017, device="cuda") for _ in range(4)]
    assert at.isdisjoint(t.data_ptr() for t in new)
    del plan, new
    new = [torch.empty(3_000_017, device="cuda") for _ in range(6)]
    assert at <= {t.data_ptr() for t in new}
