"""f8_token_logprobs and f8_token_logprobs_bwd against the definition in 64
bits: one row and many, odd vocabularies, rows that start off a 16-byte
boundary, padding that holds NaN, masked tokens (-inf and the type's lowest
value), rows without a token, ties, NaN and infinities, top k from 1 to its
limit, splits of a row over a cluster, streams, graphs and in-place calls."""
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


def _logits(rows, vocab, dtype, seed, pad=0, scale=3.0, pad_value=float("nan")):
    g = torch.Generator(device=DEV).manual_seed(seed)
    full = torch.full((rows, vocab + pad), pad_value, dtype=dtype, device=DEV)
    full[:, :vocab] = (torch.randn((rows, vocab), generator=g, device=DEV) * scale + 1.0).to(dtype)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    return full, full[:, :vocab], tokens


def _check(f8, logits, tokens, top_k, T, what):
    logp, ent, lse, ids, top = f8.f8_token_logprobs(logits, tokens, top_k=top_k, temperature=T)
    r = ref.token_logprobs(logits, tokens, T, top_k)
    keep = torch.ones_like(lse, dtype=torch.bool) if tokens is None else tokens >= 0
    ref.check(lse[keep], r["lse"][keep], r["b_lse"][keep], what + " lse")
    ref.check(ent[keep], r["entropy"][keep], r["b_entropy"][keep], what + " entropy")
    if tokens is not None:
        ref.check(logp[keep], r["logp"][keep], r["b_logp"][keep], what + " logp")
    if top_k:
        assert torch.equal(ids[keep].long(), r["top_ids"][keep]), what + " top ids"
        ref.check(top[keep], r["top_logp"][keep], r["b_top"][keep], what + " top logp")
    if tokens is not None and (~keep).any():
        assert not lse[~keep].any() and not ent[~keep].any() and not logp[~keep].any()
        if top_k:
            assert (ids[~keep] == -1).all() and (top[~keep] == NINF).all()
    return lse, ent


SHAPES = [(1, 1, 0), (2, 3, 0), (5, 7, 1), (4, 8, 0), (3, 255, 0), (9, 257, 5), (17, 1000, 8),
          (700, 512, 0), (6, 4099, 13), (1, 32768, 0), (3, 50003, 0), (2, 131072, 0), (40, 40001, 7)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_against_definition(f8, shape, dtype):
    rows, vocab, pad = shape
    _, logits, tokens = _logits(rows, vocab, dtype, rows + vocab, pad)
    for T, k in ((1.0, 0), (0.7, min(vocab, 5)), (2.0, min(vocab, 64)), (1.0, min(vocab, 256))):
        _check(f8, logits, tokens, k, T, f"{shape} {dtype} T {T} k {k}")
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_ties_and_orders(f8, dtype):
    """Equal logits go by ascending id, however they lie: all equal, two
    values, ascending, descending, -0 beside +0."""
    V = 9001
    z = torch.zeros((6, V), device=DEV)
    z[1, ::3] = 1.5
    z[2] = torch.arange(V, device=DEV) / 64
    z[3] = -torch.arange(V, device=DEV) / 64
    z[4, 1::2] = -0.0
    z[5, -5:] = 2.0
    z = z.to(dtype)
    for k in (1, 7, 256):
        _check(f8, z, None, k, 1.0, f"ties k {k}")
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("vocab", [70, 5000, 60001])
def test_masks(f8, dtype, vocab):
    _, logits, tokens = _logits(8, vocab, dtype, 3)
    logits = logits.clone()
    low = torch.finfo(dtype).min
    logits[0, ::2] = NINF
    logits[1, : vocab - 1] = NINF            # one token left
    logits[1, vocab - 1] = -3.0
    logits[2] = NINF                         # none left
    logits[3, 1:] = low                      # the type's lowest value
    logits[4] = low                          # a uniform row
    logits[5, : vocab // 2] = NINF
    tokens[6] = -1
    logits[6] = float("nan")                 # ignored: not read
    tokens[7] = -100
    # one token's entropy is 0, the uniform row's ln V
    _check(f8, logits, tokens, min(vocab, 33), 1.0, f"masks {dtype} {vocab}")
    lse, ent = _check(f8, logits[:6], tokens[:6], 0, 0.5, f"masks T {dtype} {vocab}")
    assert ent[1].item() == 0.0 and ent[2].item() == 0.0 and lse[2].item() == NINF
    assert f8.f8_last_device_status() == 0


def test_non_finite_rows(f8):
    _, logits, tokens = _logits(5, 3000, torch.bfloat16, 4)
    logits = logits.clone()
    logits[1, 2999] = float("nan")
    logits[2, 5] = float("inf")
    logits[3] = float("nan")
    logp, ent, lse, ids, top = f8.f8_token_logprobs(logits, tokens, top_k=9)
    for t in (logp, ent, lse, top):
        assert torch.isnan(t[1:4]).all() and torch.isfinite(t[0]).all() and torch.isfinite(t[4]).all()
    for r in range(5):
        assert len(set(ids[r].tolist())) == 9 and 0 <= ids[r].min() and ids[r].max() < 3000
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_NONFINITE
    assert f8.f8_last_device_status() == 0


def test_token_outside_the_vocabulary(f8):
    full, logits, tokens = _logits(4, 1000, torch.float32, 5, pad=24, pad_value=0.0)
    tokens[1] = 1000
    tokens[2] = 1 << 40
    logp, ent, lse, _, _ = f8.f8_token_logprobs(logits, tokens)
    assert torch.isnan(logp[1:3]).all() and torch.isfinite(logp[0]) and torch.isfinite(lse).all()
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_INDEX
    one = torch.ones(4, device=DEV)
    d = f8.f8_token_logprobs_bwd(logits, tokens, lse, None, one, None)
    assert torch.isfinite(d).all()
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_INDEX


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_backward(f8, shape, dtype):
    rows, vocab, pad = shape
    full, logits, tokens = _logits(rows, vocab, dtype, 2 * rows + vocab, pad)
    g = torch.Generator(device=DEV).manual_seed(6)
    if vocab > 40:
        full[0, 3:30] = NINF
        tokens[0] = 31
    if rows > 4:
        tokens[1] = -1
        full[1] = float("nan")
    a = torch.randn((rows,), generator=g, device=DEV)
    h = torch.randn((rows,), generator=g, device=DEV) * 0.3
    if rows > 4:
        a[2] = h[2] = 0.0
    for T, use in ((1.0, "both"), (0.6, "logp"), (1.7, "entropy")):
        _, ent, lse, _, _ = f8.f8_token_logprobs(logits, tokens, temperature=T)
        da, dh = (a if use != "entropy" else None), (h if use != "logp" else None)
        out = torch.full_like(full, 7.0)
        amax = torch.empty((), dtype=torch.float32, device=DEV) if dtype == torch.bfloat16 else None
        f8.f8_token_logprobs_bwd(logits, tokens, lse, ent, da, dh, temperature=T, dlogits=out,
                                 amax_out=amax)
        clean = torch.where(torch.isnan(logits), torch.zeros_like(logits), logits)
        r, b = ref.token_logprobs_bwd(clean, tokens, lse, ent, da, dh, T)
        ref.check(out[:, :vocab], r, b + ref.rounding(r, dtype) * (r != 0), f"{shape} {dtype} {use}")
        assert not out[:, vocab:].any()
        if amax is not None:
            assert amax.item() == out.float().abs().max().item()
        tight = f8.f8_token_logprobs_bwd(logits, tokens, lse, ent, da, dh, temperature=T)
        assert torch.equal(tight, out[:, :vocab])
        own = full.clone()                       # into the logits' own buffer
        f8.f8_token_logprobs_bwd(own[:, :vocab], tokens, lse, ent, da, dh, temperature=T, dlogits=own)
        assert torch.equal(own, out)
    assert f8.f8_last_device_status() == 0


def test_backward_against_differences(f8):
    V, T = 24, 0.8
    _, logits, tokens = _logits(3, V, torch.float32, 8, scale=1.0)
    g = torch.Generator(device=DEV).manual_seed(9)
    a, h = torch.randn((2, 3), generator=g, device=DEV)
    _, ent, lse, _, _ = f8.f8_token_logprobs(logits, tokens, temperature=T)
    d = f8.f8_token_logprobs_bwd(logits, tokens, lse, ent, a, h, temperature=T)

    def scalar(z):
        r = ref.token_logprobs(z, tokens, T, 0)
        return (r["logp"] * a.double() + r["entropy"] * h.double()).sum()

    z = logits.double().clone()
    num = torch.zeros_like(z)
    e = 1e-5
    for i in range(3):
        for j in range(V):
            keep = z[i, j].item()
            z[i, j] = keep + e
            up = scalar(z)
            z[i, j] = keep - e
            num[i, j] = (up - scalar(z)) / (2 * e)
            z[i, j] = keep
    # differences: e^2 times third derivatives of order 10; fp32 results of order 1
    assert (d.double() - num).abs().max().item() <= 5e-6


def test_same_bits_again_and_split_or_not(f8):
    """Equal inputs give equal bits; a row alone (split over a cluster) and
    among many (one block a row) agree within the bound."""
    _, logits, tokens = _logits(400, 33000, torch.bfloat16, 10)
    first = f8.f8_token_logprobs(logits, tokens, top_k=20)
    again = f8.f8_token_logprobs(logits, tokens, top_k=20)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    one = f8.f8_token_logprobs(logits[7:8], tokens[7:8], top_k=20)
    assert torch.equal(one[3], first[3][7:8])
    r = ref.token_logprobs(logits[7:8], tokens[7:8], 1.0, 20)
    for n, t in (("logp", one[0]), ("entropy", one[1]), ("lse", one[2])):
        ref.check(t, r[n], r["b_" + n], n)


def test_stream_and_graph(f8):
    _, logits, tokens = _logits(30, 20000, torch.bfloat16, 11)
    want = f8.f8_token_logprobs(logits, tokens, top_k=10)
    outs = [torch.zeros_like(t) for t in want]
    names = ("logp", "entropy", "lse", "top_ids", "top_logp")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f8.f8_token_logprobs(logits, tokens, top_k=10, stream=side, **dict(zip(names, outs)))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f8.f8_token_logprobs(logits, tokens, top_k=10, **dict(zip(names, outs)))
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert f8.f8_last_device_status() == 0


def test_past_2_31_elements(f8):
    V = 131072
    rows = (1 << 31) // V + 3
    big = torch.zeros((rows, V), dtype=torch.bfloat16, device=DEV)
    _, logits, tokens = _logits(3, V, torch.bfloat16, 12)
    big[-3:] = logits
    tok = torch.full((rows,), -1, dtype=torch.int64, device=DEV)
    tok[-3:] = tokens
    got = f8.f8_token_logprobs(big, tok, top_k=4)
    r = ref.token_logprobs(logits, tokens, 1.0, 4)
    assert torch.equal(got[3][-3:].long(), r["top_ids"])
    ref.check(got[2][-3:], r["lse"], r["b_lse"], "lse")
    one = torch.ones(rows, device=DEV)
    d = f8.f8_token_logprobs_bwd(big, tok, got[2], got[1], one, None, dlogits=big)
    g, b = ref.token_logprobs_bwd(logits, tokens, got[2][-3:], None, one[-3:], None, 1.0)
    ref.check(d[-3:], g, b + ref.rounding(g, torch.bfloat16), "dlogits")
    assert f8.f8_last_device_status() == 0


def test_largest_vocabulary(f8):
    V = f8.F8_MAX_VOCAB
    g = torch.Generator(device=DEV).manual_seed(13)
    for dtype in (torch.bfloat16, torch.float32):
        z = torch.randn((2, V), generator=g, device=DEV).to(dtype)
        tokens = torch.tensor([V - 1, 0], device=DEV)
        _check(f8, z, tokens, 256, 1.0, f"largest {dtype}")
    assert f8.f8_last_device_status() == 0
