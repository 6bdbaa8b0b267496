"""The distillation loss' tail class where the student leaves it next to
nothing: p_r far below fp32's normal range (and 1 - sum q a tenth) is still
the probability that the loss and the gradient are formed from, in the loss
pass, the gradient pass and the one that does both; where the tokens outside
the slots are masked, the term is dropped."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


def _confident(rows, vocab, k, pad, dtype, gap, seed):
    """Logits whose slots lie about `gap` above all others."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    full = torch.full((rows, vocab + pad), float("nan"), device=DEV)
    full[:, :vocab] = torch.randn((rows, vocab), generator=g, device=DEV) * 2.0
    ids = torch.rand((rows, vocab), generator=g, device=DEV).argsort(1)[:, :k]
    full.scatter_add_(1, ids, torch.full_like(ids, gap, dtype=torch.float32))
    values = torch.log_softmax(torch.randn((rows, k), generator=g, device=DEV), 1) + torch.log(torch.tensor(0.9))
    dloss = torch.rand((rows,), generator=g, device=DEV) + 0.5
    return full.to(dtype), ids.to(torch.int32).contiguous(), values.contiguous(), dloss


def _run(f8, full, vocab, ids, values, dloss, T, what):
    logits, dtype = full[:, :vocab], full.dtype
    r = ref.distill(logits, ids, values, T, True, dloss)
    rnd = ref.rounding(r["dlogits"], dtype) * (r["dlogits"] != 0)
    loss, lse, rest = f8.f8_distill_fwd(logits, ids, values, temperature=T, tail=True)
    ref.check(loss, r["loss"], r["b_loss"], what + " loss")
    d = f8.f8_distill_bwd(logits, ids, values, lse, rest, dloss, temperature=T, tail=True)
    ref.check(d, r["dlogits"], r["b_dlogits"] + rnd, what + " bwd")
    loss2, both = f8.f8_distill_fwd_bwd(logits, ids, values, dloss, temperature=T, tail=True)
    ref.check(loss2, r["loss"], r["b_loss"], what + " both: loss")
    ref.check(both, r["dlogits"], r["b_dlogits"] + rnd, what + " both: dlogits")
    return r, rest, both


# one block a row, a cluster a row, registers and rows walked twice, the ring
SHAPES = [(5, 300, 8, 4), (700, 640, 16, 0), (3, 70000, 24, 5), (200, 20001, 16, 7), (3, 300001, 20, 7)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gap,T", [(60.0, 1.0), (85.0, 1.0), (95.0, 1.0), (120.0, 1.0), (120.0, 0.5), (60.0, 0.2)])
def test_small_rest(f8, shape, dtype, gap, T):
    rows, vocab, k, pad = shape
    full, ids, values, dloss = _confident(rows, vocab, k, pad, dtype, gap, rows + vocab)
    r, rest, d = _run(f8, full, vocab, ids, values, dloss, T, f"{shape} {dtype} gap {gap} T {T}")
    # p_r itself, or its logarithm where fp32 does not hold it
    log_rest = torch.where(rest < 0, rest.double(), rest.double().clamp(min=1e-45).log())
    z = full[:, :vocab].double().abs().amax(1) / T
    bound = ref.K * ref.U * (2 + r["lse"].abs() + z)
    ref.check(log_rest, r["rest"].log(), bound, "rest")
    # the tail's share reaches the tokens outside the slots: q_r of dloss / T in all
    inside = torch.zeros_like(d, dtype=torch.bool).scatter_(1, ids.long(), True)
    out = torch.where(inside, torch.zeros_like(d), d).double().sum(1)
    want = -(1 - values.double().exp().sum(1)) * dloss.double() / T
    assert ((out - want).abs() <= 0.02 * want.abs() + vocab * 2.0 ** -133).all()
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("mask", [float("-inf"), -1e4, -1e9, "lowest"], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_masked_rest(f8, mask, dtype):
    """All tokens outside the slots masked: no tail term, in 64 bits too."""
    full, ids, values, dloss = _confident(4, 2003, 8, 0, dtype, 0.0, 5)
    inside = torch.zeros_like(full, dtype=torch.bool).scatter_(1, ids.long(), True)
    full[~inside] = torch.finfo(dtype).min if mask == "lowest" else mask
    _, rest, d = _run(f8, full, 2003, ids, values, dloss, 1.0, f"mask {mask}")
    assert not rest.any() and not d[~inside].any()
    assert f8.f8_last_device_status() == 0
