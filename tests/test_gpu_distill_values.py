"""Teacher values that are NaN or +inf: the row's loss and its whole gradient are
NaN, in every pass, and other rows keep theirs."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(4, 300), (4, 60001), (200, 20001)])
def test_non_finite_values(f8, rows, vocab, dtype, tail):
    g = torch.Generator(device=DEV).manual_seed(rows + vocab)
    z = (torch.randn((rows, vocab), generator=g, device=DEV) * 2).to(dtype)
    ids = torch.rand((rows, vocab), generator=g, device=DEV).argsort(1)[:, :8].to(torch.int32).contiguous()
    values = torch.log_softmax(torch.randn((rows, 8), generator=g, device=DEV), 1) - 0.1
    one = torch.ones(rows, device=DEV)
    want = f8.f8_distill_fwd_bwd(z, ids, values, one, tail=tail)
    values[1, 3], values[2, 0] = float("nan"), float("inf")
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[1:3] = True
    loss, d = f8.f8_distill_fwd_bwd(z, ids, values, one, tail=tail)
    loss2, lse, rest = f8.f8_distill_fwd(z, ids, values, tail=tail)
    d2 = f8.f8_distill_bwd(z, ids, values, lse, rest, one, tail=tail)
    for got in (loss, loss2):
        assert torch.equal(torch.isnan(got), bad)
    for got in (d, d2):
        assert torch.isnan(got[bad]).all() and torch.isfinite(got[~bad]).all()
    assert torch.equal(loss[~bad], want[0][~bad]) and torch.equal(d[~bad], want[1][~bad])
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_NONFINITE
