"""f8_distill_fwd, f8_distill_bwd and f8_distill_fwd_bwd against the definition
in 64 bits: renormalised and with the tail class, temperatures, odd and padded
vocabularies, empty slots, rows without one, equal ids, ids outside, masked
tokens, rows with zero weight, NaN, one slot to the limit, rows held in
registers and rows walked twice, in-place calls, streams and graphs."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NINF = float("-inf")


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


def _case(rows, vocab, k, dtype, tail, seed, pad=0, mass=0.9):
    g = torch.Generator(device=DEV).manual_seed(seed)
    full = torch.full((rows, vocab + pad), float("nan"), dtype=dtype, device=DEV)
    full[:, :vocab] = (torch.randn((rows, vocab), generator=g, device=DEV) * 2.0 + 0.5).to(dtype)
    ids = torch.rand((rows, vocab), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32)
    values = torch.randn((rows, k), generator=g, device=DEV) * 2.0
    if tail:
        values = torch.log_softmax(values, 1) + torch.log(torch.tensor(mass))
    dloss = torch.rand((rows,), generator=g, device=DEV) + 0.5
    return full, full[:, :vocab], ids.contiguous(), values.contiguous(), dloss


def _check(f8, full, vocab, ids, values, dloss, T, tail, what, clean=None, dx=True):
    logits = full[:, :vocab]
    r = ref.distill(logits if clean is None else clean, ids, values, T, tail, dloss)
    loss, lse, rest = f8.f8_distill_fwd(logits, ids, values, temperature=T, tail=tail)
    ref.check(loss, r["loss"], r["b_loss"], what + " loss")
    ref.check(lse, r["lse"], r["b_lse"], what + " lse")
    if tail:
        ref.check(rest, r["rest"], r["b_rest"], what + " rest")
    else:
        assert rest is None
    amax = torch.empty((), dtype=torch.float32, device=DEV) if full.dtype == torch.bfloat16 else None
    rnd = ref.rounding(r["dlogits"], full.dtype) * (r["dlogits"] != 0)
    out = torch.full_like(full, 3.0)
    f8.f8_distill_bwd(logits, ids, values, lse, rest, dloss, temperature=T, tail=tail, dlogits=out,
                      amax_out=amax)
    ref.check(out[:, :vocab], r["dlogits"], r["b_dlogits"] + rnd, what + " bwd")
    assert not out[:, vocab:].any()
    if amax is not None:
        assert amax.item() == out.float().abs().max().item()
        amax.fill_(9.0)
    both = torch.full_like(full, 3.0)
    loss2, _ = f8.f8_distill_fwd_bwd(logits, ids, values, dloss, temperature=T, tail=tail,
                                     dlogits=both, amax_out=amax)
    ref.check(loss2, r["loss"], r["b_loss"], what + " both: loss")
    ref.check(both[:, :vocab], r["dlogits"], r["b_dlogits"] + rnd, what + " both: dlogits")
    assert not both[:, vocab:].any()
    if amax is not None:
        assert amax.item() == both.float().abs().max().item()
    # the same bits again, into a tight buffer, and in place
    tight = f8.f8_distill_fwd_bwd(logits, ids, values, dloss, temperature=T, tail=tail)
    assert torch.equal(tight[0], loss2) and torch.equal(tight[1], both[:, :vocab])
    own = full.clone()
    f8.f8_distill_fwd_bwd(own[:, :vocab], ids, values, dloss, temperature=T, tail=tail, dlogits=own)
    assert torch.equal(own, both)
    own = full.clone()
    f8.f8_distill_bwd(own[:, :vocab], ids, values, lse, rest, dloss, temperature=T, tail=tail, dlogits=own)
    assert torch.equal(own, out)
    return loss, both


SHAPES = [(1, 2, 1, 0), (3, 9, 4, 3), (5, 100, 100, 4), (600, 640, 16, 0), (4, 4096, 64, 0),
          (7, 5003, 32, 13), (2, 32000, 256, 0), (3, 50003, 20, 0), (2, 131072, 64, 0),
          (300, 20001, 7, 7)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
def test_against_definition(f8, shape, dtype, tail):
    rows, vocab, k, pad = shape
    full, logits, ids, values, dloss = _case(rows, vocab, k, dtype, tail, rows + vocab, pad)
    for T in (1.0, 0.5, 2.0):
        _check(f8, full, vocab, ids, values, dloss, T, tail, f"{shape} {dtype} tail {tail} T {T}")
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("dtype,vocab", [(torch.bfloat16, 300001), (torch.float32, 140001)])
@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
def test_rows_longer_than_the_registers(f8, dtype, vocab, tail):
    full, logits, ids, values, dloss = _case(3, vocab, 50, dtype, tail, 21, 7)
    _check(f8, full, vocab, ids, values, dloss, 1.0, tail, f"long {dtype}")
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
@pytest.mark.parametrize("dtype,vocab,pad", [(torch.bfloat16, 140003, 13), (torch.bfloat16, 20480, 0),
                                             (torch.float32, 65001, 3)])
def test_many_long_rows(f8, dtype, vocab, pad, tail):
    """Several rows per SM, some of them ignored, longer than what one block
    keeps of a row."""
    full, logits, ids, values, dloss = _case(400, vocab, 40, dtype, tail, 22, pad)
    ids[5::17] = -1
    full[5::17] = float("nan")
    dloss[3::50] = 0.0
    clean = torch.where(torch.isnan(logits), torch.zeros_like(logits), logits)
    _check(f8, full, vocab, ids, values, dloss, 0.9, tail, f"many {dtype} {vocab}", clean)
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
@pytest.mark.parametrize("vocab", [300, 4001, 70000])
def test_slots_and_masks(f8, dtype, tail, vocab):
    full, logits, ids, values, dloss = _case(10, vocab, 24, dtype, tail, 31, 5)
    ids[0, 3:] = -1                              # a short list
    ids[1] = -1                                  # none: ignored, its NaN not read
    full[1] = float("nan")
    values[2, ::2] = NINF                        # empty by their value
    ids[3, 5:9] = ids[3, 4]                      # one id several times
    masked = torch.ones(vocab, dtype=torch.bool, device=DEV)
    masked[ids[4].long()] = False
    full[4, :vocab][masked] = NINF               # nothing outside the list
    full[5, :vocab] = torch.finfo(dtype).min
    full[5, ids[5, 0].long()] = 1.0              # the mask is the type's lowest value
    dloss[6] = 0.0
    full[7, ids[7, 1].long()] = 60.0             # nearly all mass on one slot
    values[8] = NINF                             # no slot by value
    full[8] = float("nan")
    if tail:
        values[9] = values[9] - values[9].exp().sum().log() + 1e-3   # sums past 1: no rest
    clean = full[:, :vocab].clone()
    clean[1] = clean[8] = 0.0
    loss, d = _check(f8, full, vocab, ids, values, dloss, 1.0, tail, f"slots {dtype} {vocab}", clean)
    assert loss[1].item() == 0.0 and loss[8].item() == 0.0
    assert not d[1].any() and not d[8].any() and not d[6].any()
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
def test_masked_targets(f8, tail):
    """A slot with mass on a masked token: infinite loss, finite gradient; a
    row of masked tokens only: infinite loss, no gradient."""
    full, logits, ids, values, dloss = _case(3, 2000, 8, torch.float32, tail, 41)
    full[0, ids[0, 2].long()] = NINF
    full[1] = NINF
    loss, d = _check(f8, full, 2000, ids, values, dloss, 1.0, tail, "masked targets")
    assert loss[0].item() == float("inf") and loss[1].item() == float("inf")
    assert torch.isfinite(d).all() and not d[1].any()
    assert f8.f8_last_device_status() == 0


def test_ids_outside_the_vocabulary(f8):
    full, logits, ids, values, dloss = _case(4, 1000, 6, torch.bfloat16, False, 42, pad=8)
    ids[1, 2] = 1000
    ids[2, 0] = 2 ** 31 - 1
    clean = ids.clone()
    clean[clean >= 1000] = -1
    got = f8.f8_distill_fwd_bwd(logits, ids, values, dloss)
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_INDEX
    want = f8.f8_distill_fwd_bwd(logits, clean, values, dloss)
    assert f8.f8_last_device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    _, lse, _ = f8.f8_distill_fwd(logits, ids, values)
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_INDEX
    d = f8.f8_distill_bwd(logits, ids, values, lse, None, dloss)
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_INDEX
    assert torch.isfinite(d).all()


@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
def test_non_finite_rows(f8, tail):
    full, logits, ids, values, dloss = _case(4, 3000, 6, torch.bfloat16, tail, 43)
    full[1, 77] = float("nan")
    full[2, ids[2, 0].long()] = float("inf")
    loss, lse, rest = f8.f8_distill_fwd(logits, ids, values, tail=tail)
    assert torch.isnan(loss[1:3]).all() and torch.isfinite(loss[0]) and torch.isfinite(loss[3])
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_NONFINITE
    loss, d = f8.f8_distill_fwd_bwd(logits, ids, values, dloss, tail=tail)
    assert torch.isnan(loss[1:3]).all() and torch.isnan(d[1:3]).any(1).all()
    assert torch.isfinite(d[0]).all() and torch.isfinite(d[3]).all()
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_NONFINITE


def test_gradient_against_differences(f8):
    V, k, T = 20, 5, 1.3
    for tail in (False, True):
        full, logits, ids, values, dloss = _case(3, V, k, torch.float32, tail, 44)
        ids[1, 3] = ids[1, 2]
        _, d = f8.f8_distill_fwd_bwd(logits, ids, values, dloss, temperature=T, tail=tail)
        z = logits.double().clone()
        num = torch.zeros_like(z)
        e = 1e-5

        def scalar():
            return (ref.distill(z, ids, values, T, tail, dloss)["loss"] * dloss.double()).sum()

        for i in range(3):
            for j in range(V):
                keep = z[i, j].item()
                z[i, j] = keep + e
                up = scalar()
                z[i, j] = keep - e
                num[i, j] = (up - scalar()) / (2 * e)
                z[i, j] = keep
        # differences: e^2 times third derivatives of order 10; fp32 results of order 1
        assert (d.double() - num).abs().max().item() <= 5e-6


def test_a_teacher_with_the_students_own_logits_has_no_loss(f8):
    """The tail loss of a model against its own top log probabilities is 0,
    and so is its gradient, up to rounding."""
    g = torch.Generator(device=DEV).manual_seed(45)
    z = (torch.randn((20, 30000), generator=g, device=DEV) * 3).to(torch.bfloat16)
    for T in (1.0, 0.7):
        _, _, _, ids, top = f8.f8_token_logprobs(z, top_k=64, temperature=T)
        one = torch.ones(20, device=DEV)
        loss, d = f8.f8_distill_fwd_bwd(z, ids, top, one, temperature=T, tail=True)
        # sums of 64 terms of order 1 whose fp32 errors cancel to first order
        assert loss.abs().max().item() <= 2e-5
        assert d.float().abs().max().item() <= 2e-5


def test_stream_and_graph(f8):
    full, logits, ids, values, dloss = _case(30, 20000, 16, torch.bfloat16, True, 46)
    want = f8.f8_distill_fwd_bwd(logits, ids, values, dloss, tail=True)
    loss, d = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f8.f8_distill_fwd_bwd(logits, ids, values, dloss, tail=True, loss=loss, dlogits=d, stream=side)
    side.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(d, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f8.f8_distill_fwd_bwd(logits, ids, values, dloss, tail=True, loss=loss, dlogits=d)
    loss.zero_()
    d.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(d, want[1])
    assert f8.f8_last_device_status() == 0


def test_past_2_31_elements(f8):
    V = 131072
    rows = (1 << 31) // V + 3
    big = torch.zeros((rows, V), dtype=torch.bfloat16, device=DEV)
    full, logits, ids, values, dloss = _case(3, V, 16, torch.bfloat16, False, 47)
    big[-3:] = logits
    all_ids = torch.full((rows, 16), -1, dtype=torch.int32, device=DEV)
    all_ids[-3:] = ids
    all_values = torch.zeros((rows, 16), device=DEV)
    all_values[-3:] = values
    w = torch.ones(rows, device=DEV)
    w[-3:] = dloss
    r = ref.distill(logits, ids, values, 1.0, False, dloss)
    loss, d = f8.f8_distill_fwd_bwd(big, all_ids, all_values, w, dlogits=big)
    ref.check(loss[-3:], r["loss"], r["b_loss"], "loss")
    ref.check(d[-3:], r["dlogits"], r["b_dlogits"] + ref.rounding(r["dlogits"], torch.bfloat16), "dlogits")
    assert not d[:-3:1024].any()
    assert f8.f8_last_device_status() == 0
