"""f8_rope against the rotation in 64 bits (tests/block_reference.py): both
layouts, both types, whole and part heads of even and odd sizes, queries with and
without keys, packed and transposed tensors, far positions, padding rows, in
place; the inverse as the gradient, streams and captured calls."""
import pytest
import torch

import block_reference as ref
from ops_reference import check, rounding

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


def _rnd(shape, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _check(f8, x, got, pos, freqs, scale, layout, inverse, what):
    if x.dim() == 3:
        x, got, pos = x[None], got[None], pos.reshape(1, -1)
    pos = pos.expand(x.shape[:2])
    want, bound = ref.rope(x, pos, freqs, scale, layout == f8.F8_ROPE_INTERLEAVED, inverse)
    # a column that is copied is exact
    bound = torch.where(bound > 0, bound + rounding(want, x.dtype), bound)
    check(got, want, bound, what)


# (tokens, q heads, k heads, dim, rot)
SHAPES = [(1, 1, 1, 2, 2), (3, 2, 1, 6, 4), (5, 3, 1, 64, 64), (8, 32, 8, 128, 128), (17, 4, 2, 80, 20), (9, 5, 5, 96, 24),
          (40, 8, 1, 128, 96), (33, 7, 3, 72, 48), (6, 2, 2, 256, 64), (130, 16, 4, 64, 32), (2, 1, 1, 1024, 1024),
          (5, 40, 8, 255, 254), (1000, 3, 1, 192, 96), (4, 3, 2, 100, 36)]


@pytest.mark.parametrize("layout", [0, 1], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(f8, shape, dtype, layout):
    n, hq, hk, dim, rot = shape
    q, k = _rnd((n, hq, dim), 1, dtype), _rnd((n, hk, dim), 2, dtype)
    freqs = f8.f8_rope_frequencies(rot, 500000.0, device=DEV)
    pos = torch.randint(0, 5000, (n,), device=DEV)
    pos[0] = 0
    for inverse in (False, True):
        qo, ko = f8.f8_rope(q, pos, freqs, k=k, layout=layout, scale=1.25, inverse=inverse)
        _check(f8, q, qo, pos, freqs, 1.25, layout, inverse, "q")
        _check(f8, k, ko, pos, freqs, 1.25, layout, inverse, "k")
        alone, none = f8.f8_rope(q, pos, freqs, layout=layout, scale=1.25, inverse=inverse)
        assert none is None and torch.equal(alone, qo)
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_views(f8, layout, dtype):
    """Columns of a packed projection, heads ahead of the sequence, an offset start, and outputs of other strides."""
    b, s, hq, hk, dim = 3, 37, 8, 2, 64
    freqs = f8.f8_rope_frequencies(48, device=DEV)
    pos = torch.randint(0, 999, (b, s), device=DEV)
    packed = _rnd((b, s, hq + 2 * hk, dim), 3, dtype)
    before = packed.clone()
    q, k = packed[:, :, :hq], packed[:, :, hq:hq + hk]
    qo, ko = f8.f8_rope(q, pos, freqs, k=k, layout=layout)
    _check(f8, q, qo, pos, freqs, 1.0, layout, False, "q")
    _check(f8, k, ko, pos, freqs, 1.0, layout, False, "k")
    assert torch.equal(packed, before)
    f8.f8_rope(q, pos, freqs, k=k, layout=layout, q_out=q, k_out=k)      # in place, and nothing else
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(packed[:, :, hq + hk:], before[:, :, hq + hk:])
    heads_first = before[:, :, :hq].transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.empty((b, hq, s, dim), dtype=dtype, device=DEV).transpose(1, 2)
    got, _ = f8.f8_rope(heads_first, pos, freqs, layout=layout, q_out=out)
    assert got is out and torch.equal(out, qo)
    odd = torch.empty((b, s, hq, dim + 1), dtype=dtype, device=DEV)[..., 1:]   # rows that no vector fits
    odd.copy_(before[:, :, :hq])
    assert torch.equal(f8.f8_rope(odd, pos, freqs, layout=layout)[0], qo)
    broad = before[:, :, :1].expand(b, s, hq, dim)                             # one head read by all
    assert torch.equal(f8.f8_rope(broad, pos, freqs, layout=layout)[0][:, :, 3],
                       f8.f8_rope(before[:, :, :1], pos, freqs, layout=layout)[0][:, :, 0])


def test_position_forms(f8):
    """[seq] for the whole batch, a strided list, and [batch, seq]."""
    q = _rnd((4, 9, 2, 32), 4, BF)
    freqs = f8.f8_rope_frequencies(32, device=DEV)
    pos = torch.arange(9, device=DEV) * 3 + 7
    want, _ = f8.f8_rope(q, pos.expand(4, 9).contiguous(), freqs)
    assert torch.equal(f8.f8_rope(q, pos, freqs)[0], want)
    assert torch.equal(f8.f8_rope(q, pos.expand(4, 9), freqs)[0], want)
    spread = torch.zeros(18, dtype=torch.int64, device=DEV)
    spread[::2] = pos
    assert torch.equal(f8.f8_rope(q, spread[::2], freqs)[0], want)
    flat, _ = f8.f8_rope(q.reshape(36, 2, 32), pos.repeat(4), freqs)
    assert torch.equal(flat.reshape(want.shape), want)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_far_positions(f8, layout, dtype):
    """Angles of some 2^30 positions stay those of 64 bits: the frequency's rounding there, 2^30 * 2^-53 radians, is far
    below the outputs' own."""
    pos = torch.tensor([0, 1, 131071, 1 << 20, (1 << 30) + 12345, (1 << 31) + 1], device=DEV)
    x = _rnd((6, 2, 64), 5, dtype)
    freqs = f8.f8_rope_frequencies(64, device=DEV)
    got, _ = f8.f8_rope(x, pos, freqs, layout=layout)
    _check(f8, x, got, pos, freqs, 1.0, layout, False, "far")
    assert torch.equal(got[0], x[0])


def test_padding_rows(f8):
    x = _rnd((2, 12, 3, 64), 6, BF)
    freqs = f8.f8_rope_frequencies(64, device=DEV)
    pos = torch.arange(12, device=DEV).repeat(2, 1)
    pos[0, 7:] = -1
    pos[1] = -9
    got, _ = f8.f8_rope(x, pos, freqs, scale=3.0)
    _check(f8, x, got, pos, freqs, 3.0, 0, False, "padding")
    assert torch.equal(got[0, 7:], x[0, 7:]) and torch.equal(got[1], x[1])
    x[0, 9] = float("nan")
    got, _ = f8.f8_rope(x, pos, freqs)
    assert torch.isnan(got).sum() == 3 * 64


@pytest.mark.parametrize("layout", [0, 1])
def test_inverse_is_the_gradient(f8, layout):
    """<dy, rope(x)> = <rope_inverse(dy), x>, and against differences: the call is linear."""
    x, dy = _rnd((50, 4, 96), 7, torch.float32), _rnd((50, 4, 96), 8, torch.float32)
    pos = torch.randint(0, 4000, (50,), device=DEV)
    freqs = f8.f8_rope_frequencies(64, device=DEV)
    call = lambda v, inverse=False: f8.f8_rope(v, pos, freqs, layout=layout, scale=1.3, inverse=inverse)[0].double()  # noqa: E731
    g = call(dy, True)
    # each of the 19200 products is within 2^-20 of its size
    size = (dy.double().abs() * call(x).abs()).sum() + (g.abs() * x.double().abs()).sum()
    assert ((dy.double() * call(x)).sum() - (g * x.double()).sum()).abs() <= 2.0 ** -20 * size
    d = _rnd(x.shape, 9, torch.float32)
    diff = (dy.double() * (call(x + d) - call(x - d)) / 2).sum()
    assert (diff - (g * d.double()).sum()).abs() <= 2.0 ** -18 * (dy.double().abs() * (x.double().abs() + d.double().abs())).sum() * 2.6


def test_round_trip(f8):
    x = _rnd((64, 8, 128), 10, torch.float32)
    pos = torch.arange(64, device=DEV)
    freqs = f8.f8_rope_frequencies(128, device=DEV)
    y, _ = f8.f8_rope(x, pos, freqs)
    back, _ = f8.f8_rope(y, pos, freqs, inverse=True)
    assert (back - x).abs().max() <= 2.0 ** -19 * x.abs().max()


def test_captured_and_streams(f8):
    q, k = _rnd((600, 8, 128), 11, BF), _rnd((600, 2, 128), 12, BF)
    pos = torch.arange(600, device=DEV)
    freqs = f8.f8_rope_frequencies(128, device=DEV)
    want = f8.f8_rope(q, pos, freqs, k=k)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        f8.f8_rope(q, pos, freqs, k=k, q_out=qo, k_out=ko)
    for _ in range(2):
        qo.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    pos.add_(5)   # a captured call reads the positions of its replay
    graph.replay()
    assert torch.equal(qo, f8.f8_rope(q, pos, freqs)[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = f8.f8_rope(q, pos, freqs, k=k, stream=side)
    side.synchronize()
    assert torch.equal(got[0], qo) and torch.equal(got[1], f8.f8_rope(k, pos, freqs)[0])


def test_empty(f8):
    freqs = f8.f8_rope_frequencies(64, device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    assert f8.f8_rope(torch.zeros((0, 4, 64), dtype=BF, device=DEV), none, freqs)[0].shape == (0, 4, 64)
    q = torch.zeros((3, 0, 64), dtype=BF, device=DEV)
    k = _rnd((3, 2, 64), 13, BF)
    pos = torch.arange(3, device=DEV)
    _, ko = f8.f8_rope(q, pos, freqs, k=k)
    assert torch.equal(ko, f8.f8_rope(k, pos, freqs)[0])


def test_past_2_31_elements(f8):
    """Offsets of a long cache: rows whose elements lie past 2^31."""
    n, h, d = 1 << 18, 66, 128
    x = torch.zeros((n, h, d), dtype=BF, device=DEV)
    x[-1] = _rnd((h, d), 14, BF)
    pos = torch.zeros(n, dtype=torch.int64, device=DEV)
    pos[-1] = 77
    freqs = f8.f8_rope_frequencies(d, device=DEV)
    want, _ = f8.f8_rope(x[-1:].clone(), pos[-1:], freqs)
    got, _ = f8.f8_rope(x, pos, freqs, q_out=x)
    assert x.numel() > 1 << 31 and torch.equal(got[-1:], want) and not got[:-1].any()


@pytest.mark.parametrize("layout", [0, 1], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim, rot", [(64, 64), (64, 48), (20, 12)])
def test_frequencies_that_are_no_numbers(f8, layout, dtype, dim, rot):
    """A pair whose frequency is NaN or infinite is NaN at every position, as sine and cosine of its angle are, 0 times
    infinity among them; the other pairs and rows of padding are as they are without it.  The largest finite frequency
    and the smallest turn by a number."""
    x = _rnd((7, 3, dim), 15, dtype)
    pos = torch.tensor([0, 1, 5, -1, 900, 1 << 40, 3], device=DEV)
    freqs = f8.f8_rope_frequencies(rot, device=DEV)
    half = rot // 2
    for inverse in (False, True):
        want, _ = f8.f8_rope(x, pos, freqs, layout=layout, inverse=inverse)
        bad = freqs.clone()
        bad[1], bad[half - 2], bad[half - 1] = float("nan"), float("inf"), float("-inf")
        got, _ = f8.f8_rope(x, pos, bad, layout=layout, inverse=inverse)
        gone = torch.zeros(dim, dtype=torch.bool, device=DEV)
        for i in (1, half - 2, half - 1):
            gone[[i, i + half] if layout == 0 else [2 * i, 2 * i + 1]] = True
        assert torch.equal(got[:, :, ~gone], want[:, :, ~gone])
        rows = pos >= 0
        assert torch.isnan(got[rows][:, :, gone]).all() and torch.equal(got[~rows], x[~rows])
        ends = freqs.clone()
        ends[1], ends[half - 1] = 1.7e308, 5e-324
        assert torch.isfinite(f8.f8_rope(x, pos, ends, layout=layout, inverse=inverse)[0]).all()


def test_empty_views(f8):
    """Views of packed rows without a batch, rows or heads: their strides are those of no output, and of no account."""
    freqs = f8.f8_rope_frequencies(64, device=DEV)
    for b, s in ((0, 5), (2, 0), (0, 0)):
        packed = torch.zeros((b, s, 12, 64), dtype=BF, device=DEV)
        pos = torch.zeros((b, s), dtype=torch.int64, device=DEV)
        for inverse in (False, True):
            q, k = f8.f8_rope(packed[:, :, :8], pos, freqs, k=packed[:, :, 8:10], inverse=inverse)
            assert q.shape == (b, s, 8, 64) and k.shape == (b, s, 2, 64)
    packed = _rnd((2, 5, 12, 64), 16, BF)
    pos = torch.arange(5, device=DEV)
    q, k = f8.f8_rope(packed[:, :, 3:3], pos, freqs, k=packed[:, :, 8:10])  # no queries
    assert q.shape == (2, 5, 0, 64) and torch.equal(k, f8.f8_rope(packed[:, :, 8:10], pos, freqs)[0])
    assert f8.f8_last_device_status() == 0


def test_in_place_single_rows(f8):
    """In place where a dimension is of one: the strides that no element goes by may differ."""
    packed = _rnd((1, 5, 12, 64), 17, BF)
    pos, freqs = torch.arange(5, device=DEV), f8.f8_rope_frequencies(64, device=DEV)
    q = packed[:, :, :8]
    want, _ = f8.f8_rope(q, pos, freqs)
    out = q.as_strided(q.shape, (7, *q.stride()[1:]), q.storage_offset())
    f8.f8_rope(q, pos, freqs, q_out=out)
    assert torch.equal(q, want)
