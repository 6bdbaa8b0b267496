"""The operators between a block's linears on inputs without rows: outputs that are
sums over the rows are 0, whatever the memory held, and nothing else is refused that
is taken with rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


def _poison(n=64):
    """Memory that the allocator hands out next holds ones."""
    blocks = [torch.full((n, 256), 1.0, dtype=BF, device=DEV) for _ in range(16)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("side", [False, True])
def test_one_gate_of_no_rows(f8, side):
    none = torch.zeros((0, 64), dtype=BF, device=DEV)
    w, stats = torch.ones(64, dtype=BF, device=DEV), torch.zeros((4, 0), device=DEV)
    _poison(1)
    dgate = torch.full((64,), 5.0, dtype=torch.float32, device=DEV)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if side else None
    kw = dict(w_post=w, gate=w.float(), kind=f8.F8_LAYER_NORM, stream=stream)
    given = f8.f8_residual_norm_bwd(none, None, none, none, w, stats, dgate=dgate, **kw)
    new = f8.f8_residual_norm_bwd(none, None, none, none, w, stats, **kw)
    torch.cuda.synchronize()
    assert given[6] is dgate and not dgate.any()
    assert new[6].shape == (64,) and all(not t.any() for t in new[2:])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("lead, gate", [((0,), (64,)), ((0,), (0, 64)), ((0, 5), (64,)), ((0, 5), (0, 64)),
                                        ((0, 5), (0, 1, 64)), ((3, 0), (3, 64)), ((3, 0), (3, 0, 64))])
def test_gated_norm_of_no_rows(f8, lead, gate, kind):
    from float8_mixed_precision_gb300 import nn
    m = nn.ResidualNorm(64, kind=kind, device=DEV)
    a, r, g = (torch.ones(s, dtype=BF, device=DEV).requires_grad_(True) for s in ((*lead, 64), (*lead, 64), gate))
    _poison(1)
    r_out, y = m(a, r, g)
    assert r_out.shape == y.shape == (*lead, 64)
    (r_out.float().sum() + y.float().sum()).backward()
    for t in (a, r, g, *m.parameters()):
        assert t.grad.shape == t.shape and not t.grad.any()
    assert f8.f8_last_device_status() == 0
