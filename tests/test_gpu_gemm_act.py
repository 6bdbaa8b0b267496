"""f8_gemm_act and f8_act_bwd against the definitions in 64 bits
(tests/block_reference.py): every activation, bias type and format, with and
without residual and kept input; sizes on every kernel path, one row, odd widths;
far values of every activation, infinities and NaN; in-place calls, the amax,
streams, captured calls, and the bias's gradient in a fixed order."""
import math

import pytest
import torch

import block_reference as ref
from ops_reference import check, rounding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
CODES = {0: (torch.float8_e4m3fn, 448.0), 1: (torch.float8_e5m2, 57344.0)}


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


def _act(f8, name):
    return getattr(f8, "F8_ACT_" + name.upper())


def _codes(shape, std, fmt, gen):
    code, most = CODES[fmt]
    x = torch.randn(shape, generator=gen, device=DEV) * std
    s = (most / x.abs().amax()).reshape(1)
    return (x * s).clamp(-most, most).to(code).view(torch.uint8), s


def _inputs(M, N, K, seed, fa=0, fb=0, bias=BF):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    a, sa = _codes((M, K), 1.0, fa, gen)
    b, sb = _codes((N, K), 1.6 / math.sqrt(K), fb, gen)
    bias = None if bias is None else (torch.randn((N,), generator=gen, device=DEV) * 0.5).to(bias)
    res = torch.randn((M, N), generator=gen, device=DEV).to(BF)
    return a, sa, b, sb, bias, res


def _check(f8, M, N, K, act, seed, fa=0, fb=0, bias=BF, residual=True, keep=True, amax=True):
    a, sa, b, sb, bias, res = _inputs(M, N, K, seed, fa, fb, bias)
    res = res if residual else None
    top = torch.full((), -1.0, device=DEV) if amax else None
    y, z = f8.f8_gemm_act(a, b, sa, sb, bias=bias, act=_act(f8, act), residual=res, want_z=keep, amax_out=top,
                          fmt_a=fa, fmt_b=fb)
    inv = 1.0 / (sa.double() * sb.double())
    rz, ry, bz, by = ref.gemm_act(a.view(CODES[fa][0]).double(), b.view(CODES[fb][0]).double(), inv, bias, act, res)
    what = f"{M}x{N}x{K} {act}"
    check(y, ry, by + rounding(ry, BF), what + " y")
    assert (z is not None) == keep
    if keep:
        check(z, rz, bz + rounding(rz, BF), what + " z")
    if amax:
        assert top.item() == y.float().abs().max().item()
    assert f8.f8_last_device_status() == 0


# (M, N, K): few rows, one row, the edges of the tiles, odd widths, one K block and less
SHAPES = [(1, 1, 16), (1, 256, 128), (8, 4096, 512), (16, 48, 64), (33, 130, 144), (64, 1000, 2048), (65, 264, 256),
          (127, 129, 272), (128, 512, 128), (200, 1001, 208), (255, 8, 96), (256, 256, 128), (257, 2056, 160),
          (300, 77, 1040), (1000, 5003, 64), (2048, 520, 4096)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_shapes(f8, shape, act):
    _check(f8, *shape, act, seed=hash(shape) % 1000)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M, N", [(9, 264), (300, 520), (40, 33), (290, 131)])
def test_activations(f8, act, M, N):
    _check(f8, M, N, 256, act, seed=5)


@pytest.mark.parametrize("fa", [0, 1])
@pytest.mark.parametrize("fb", [0, 1])
@pytest.mark.parametrize("M", [24, 272])
def test_formats(f8, fa, fb, M):
    _check(f8, M, 320, 512, "gelu_tanh", seed=7, fa=fa, fb=fb)


@pytest.mark.parametrize("bias", [None, BF, torch.float32])
@pytest.mark.parametrize("residual, keep, amax", [(False, False, False), (True, False, True), (False, True, True),
                                                  (True, True, False)])
@pytest.mark.parametrize("M, N", [(12, 392), (400, 392), (12, 391), (400, 391)])
def test_parts(f8, bias, residual, keep, amax, M, N):
    _check(f8, M, N, 144, "silu", seed=11, bias=bias, residual=residual, keep=keep, amax=amax)


def test_many_tiles(f8):
    """More tiles than the persistent blocks take at once."""
    _check(f8, 2304, 6400, 128, "gelu_tanh", seed=13)


@pytest.mark.parametrize("M, N", [(24, 264), (520, 264), (24, 65), (520, 65)])
def test_residual_in_place(f8, M, N):
    a, sa, b, sb, bias, res = _inputs(M, N, 256, 17)
    want, _ = f8.f8_gemm_act(a, b, sa, sb, bias=bias, act=f8.F8_ACT_SILU, residual=res)
    y, _ = f8.f8_gemm_act(a, b, sa, sb, bias=bias, act=f8.F8_ACT_SILU, residual=res, y=res)
    assert y is res and torch.equal(y, want)


@pytest.mark.parametrize("M, N", [(320, 5002), (513, 1003), (300, 66), (4100, 193), (3000, 2001)])
def test_rows_off_vectors(f8, M, N):
    """Rows that start anywhere in 16 bytes, over several rounds of tiles: every output, what lies around it, and
    the residual in place."""
    _check(f8, M, N, 80, "gelu", M + N)
    a, sa, b, sb, bias, res = _inputs(M, N, 80, 3)
    kw = dict(bias=bias, act=f8.F8_ACT_SILU)
    want, z = f8.f8_gemm_act(a, b, sa, sb, residual=res, want_z=True, **kw)
    around = 64
    flat = [torch.full((M * N + 2 * around,), 7.0, dtype=BF, device=DEV) for _ in range(2)]
    y2, z2 = (f[around:around + M * N].view(M, N) for f in flat)
    y2.copy_(res)
    f8.f8_gemm_act(a, b, sa, sb, residual=y2, y=y2, z=z2, **kw)
    assert torch.equal(y2, want) and torch.equal(z2, z)
    for f in flat:
        assert (f[:around] == 7.0).all() and (f[around + M * N:] == 7.0).all()


@pytest.mark.parametrize("M, N", [(24, 264), (520, 264), (24, 65), (520, 65)])
def test_plain_equals_f8_gemm(f8, M, N):
    a, sa, b, sb, _, _ = _inputs(M, N, 512, 19)
    y, _ = f8.f8_gemm_act(a, b, sa, sb)
    assert (y.float() - f8.f8_gemm(a, b, sa, sb).float()).abs().max() <= 2 ** -7 * y.float().abs().max()


@pytest.mark.parametrize("M", [5, 300])
def test_empty(f8, M):
    a, sa, b, sb, _, _ = _inputs(M, 64, 64, 23)
    top = torch.full((), 3.0, device=DEV)
    assert f8.f8_gemm_act(a[:0], b, sa, sb, amax_out=top)[0].shape == (0, 64) and top.item() == 0
    assert f8.f8_gemm_act(a, b[:0], sa, sb)[0].shape == (M, 0)


@pytest.mark.parametrize("M, N", [(16, 256), (512, 256), (16, 255)])
def test_nonfinite_y(f8, M, N):
    """An infinite residual reaches its own element only, and the status."""
    a, sa, b, sb, bias, res = _inputs(M, N, 128, 29)
    want, _ = f8.f8_gemm_act(a, b, sa, sb, bias=bias, residual=res)
    res[3, 7] = float("inf")
    top = torch.zeros((), device=DEV)
    y, _ = f8.f8_gemm_act(a, b, sa, sb, bias=bias, residual=res, amax_out=top)
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_NONFINITE
    assert y[3, 7] == float("inf")
    y[3, 7] = want[3, 7]
    assert torch.equal(y, want)


@pytest.mark.parametrize("M, N", [(16, 1024), (512, 1024), (96, 333)])
def test_captured(f8, M, N):
    a, sa, b, sb, bias, res = _inputs(M, N, 512, 31)
    kw = dict(bias=bias, act=f8.F8_ACT_GELU, residual=res, want_z=True)
    want = f8.f8_gemm_act(a, b, sa, sb, **kw)
    y, z, top = torch.zeros_like(want[0]), torch.zeros_like(want[0]), torch.zeros((), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f8.f8_gemm_act(a, b, sa, sb, y=y, z=z, amax_out=top, **kw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f8.f8_gemm_act(a, b, sa, sb, y=y, z=z, amax_out=top, **kw)
    y.zero_(), z.zero_()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])
        assert top.item() == y.float().abs().max().item()


def test_two_at_once(f8):
    """Calls on two streams share nothing."""
    sets = [_inputs(24, 4096, 2048, 37), _inputs(640, 1024, 512, 41)]
    call = lambda s, st=None: f8.f8_gemm_act(s[0], s[2], s[1], s[3], bias=s[4], act=f8.F8_ACT_SILU,  # noqa: E731
                                             residual=s[5], stream=st)[0]
    want = [call(s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[call(s, st) for s, st in zip(sets, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


# ---------------------------------------------------------------- backward
BWD = [(1, 1), (1, 8), (3, 255), (31, 256), (33, 264), (64, 1000), (257, 1001), (700, 4104), (2000, 96), (5, 30001),
       (4099, 520)]


@pytest.mark.parametrize("shape", BWD, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act", ref.ACTS)
def test_bwd(f8, shape, act):
    gen = torch.Generator(device=DEV).manual_seed(43)
    z = (torch.randn(shape, generator=gen, device=DEV) * 2).to(BF)
    dy = (torch.randn(shape, generator=gen, device=DEV) * 0.01).to(BF)
    rdz, rdb, bdz, bdb = ref.act_bwd(dy, z, act)
    for dtype in (BF, torch.float32):
        top = torch.zeros((), device=DEV)
        dz, db = f8.f8_act_bwd(dy, None if act == "none" else z, _act(f8, act), bias_dtype=dtype, amax_out=top)
        check(dz, rdz, bdz + rounding(rdz, BF), f"{shape} {act} dz")
        check(db, rdb, bdb + rounding(rdb, dtype), f"{shape} {act} dbias")
        assert top.item() == dz.float().abs().max().item()
    again = f8.f8_act_bwd(dy, z, _act(f8, act), bias_dtype=torch.float32)
    assert torch.equal(again[1], db) and torch.equal(again[0], dz)
    alone = f8.f8_act_bwd(dy, z, _act(f8, act), bias_dtype=torch.float32, want_dz=False)
    assert alone[0] is None and torch.equal(alone[1], db)
    alone = f8.f8_act_bwd(dy, z, _act(f8, act), want_dbias=False)
    assert alone[1] is None and torch.equal(alone[0], dz)
    inplace = dy.clone()
    f8.f8_act_bwd(inplace, z, _act(f8, act), dz=inplace)
    assert torch.equal(inplace, dz)
    assert f8.f8_last_device_status() == 0


def _every_bf16():
    """Every finite bf16 value, as [rows, 256]."""
    bits = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(BF)
    return bits[torch.isfinite(bits)].reshape(-1, 256)


@pytest.mark.parametrize("act", ref.ACTS[1:])
def test_bwd_every_value(f8, act):
    z = _every_bf16()
    dy = torch.ones_like(z)
    dz, _ = f8.f8_act_bwd(dy, z, _act(f8, act), want_dbias=False)
    near = z.double().clamp(-2.0 ** 40, 2.0 ** 40) if act != "relu2" else z.double()
    rdz, _, bdz, _ = ref.act_bwd(dy, near, act)
    # past 2^40 the slopes are constants; values below 2^-119 may come out as 0
    # (a reciprocal below fp32's normal range, 2^-126, times |z| < 89).  Past |z| = 16 what is left of the
    # bound is relative to the value: 16 steps as in act_steps, and SiLU's exponent on the negative side, v = |z| log2 e,
    # whose rounding and whose factor's (2^-24 v and 2^-26 v) give exp a relative error of 1.44 * 1.25 * ln 2 * |z| 2^-24
    bdz = torch.where(z.abs() > 16, (16 + 0.63 * z.double().abs()) * 2.0 ** -23 * rdz.abs(), bdz)
    check(dz, rdz, bdz + rounding(rdz, BF) + 2.0 ** -119, act)


@pytest.mark.parametrize("act", ref.ACTS[1:])
def test_value_at_every_bias(f8, act):
    """The activation of every finite bf16 value, which the bias brings: the products are 0."""
    z = _every_bf16().reshape(-1)
    a, b = torch.zeros((2, 16), dtype=torch.uint8, device=DEV), torch.zeros((z.numel(), 16), dtype=torch.uint8, device=DEV)
    one = torch.ones(1, device=DEV)
    y, kept = f8.f8_gemm_act(a, b, one, one, bias=z, act=_act(f8, act), want_z=True)
    assert torch.equal(kept, z.expand(2, -1)) and torch.equal(y[0], y[1])
    zd = z.double()
    want = ref.act(act, zd)
    steps = torch.where(zd.abs() > 16, 16.0 + 0.63 * zd.abs(), ref.act_steps(zd))   # as in the test above
    check(y[0], want, steps * 2.0 ** -23 * want.abs() + rounding(want, BF) + 2.0 ** -119, act)


@pytest.mark.parametrize("act", ref.ACTS)
def test_nan_passes(f8, act):
    z = torch.zeros((4, 64), dtype=BF, device=DEV)
    z[1, 5] = float("nan")
    top = torch.zeros((), device=DEV)
    dy = torch.ones_like(z)
    if act == "none":
        dy[1, 5] = float("nan")
    dz, db = f8.f8_act_bwd(dy, z, _act(f8, act), amax_out=top)
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_NONFINITE
    bad = torch.isnan(dz)
    assert bad[1, 5] and bad.sum() == 1 and torch.isnan(db[5]) and torch.isnan(db).sum() == 1
    a, b, one = torch.zeros((2, 16), dtype=torch.uint8, device=DEV), torch.zeros((64, 16), dtype=torch.uint8, device=DEV), torch.ones(1, device=DEV)
    y, _ = f8.f8_gemm_act(a, b, one, one, bias=z[1], act=_act(f8, act))
    assert torch.isnan(y[:, 5]).all() and torch.isnan(y).sum() == 2


@pytest.mark.parametrize("shape", [(40, 9), (40, 131), (300, 1001), (70, 5003)])
def test_bwd_neighbours_of_odd_rows(f8, shape):
    """NaN and infinities at a row's ends reach their own columns' sums only, and no other row."""
    gen = torch.Generator(device=DEV).manual_seed(53)
    z, dy = (torch.randn(shape, generator=gen, device=DEV).to(BF) for _ in range(2))
    dz, db = f8.f8_act_bwd(dy, z, f8.F8_ACT_SILU)
    dirty = dy.clone()
    dirty[3, -1], dirty[11, 0], dirty[26, -1] = float("nan"), float("inf"), float("-inf")
    got, gb = f8.f8_act_bwd(dirty, z, f8.F8_ACT_SILU)
    same = torch.isfinite(dirty)
    assert torch.equal(got[same], dz[same]) and not torch.isfinite(got[~same]).any()
    assert torch.equal(gb[1:-1], db[1:-1]) and not torch.isfinite(gb[[0, -1]]).any()


@pytest.mark.parametrize("act", ref.ACTS[1:])
def test_bwd_against_differences(f8, act):
    """The slope against differences of the forward call's own values, whose inputs a bias in 32 bits brings; at points
    where both sides of the difference lie on one side of 0."""
    n, h = 512, 2.0 ** -6
    z = torch.linspace(-4.0, 4.0, n, device=DEV).to(BF)
    z = torch.where(z.abs() < 0.1, torch.full_like(z, 0.125), z)
    a, b, one = torch.zeros((1, 16), dtype=torch.uint8, device=DEV), torch.zeros((n, 16), dtype=torch.uint8, device=DEV), torch.ones(1, device=DEV)
    up, _ = f8.f8_gemm_act(a, b, one, one, bias=z.float() + h, act=_act(f8, act))
    down, _ = f8.f8_gemm_act(a, b, one, one, bias=z.float() - h, act=_act(f8, act))
    dz, _ = f8.f8_act_bwd(torch.ones((1, n), dtype=BF, device=DEV), z[None], _act(f8, act), want_dbias=False)
    got = (up[0].double() - down[0].double()) / (2 * h)
    # the outputs' rounding (half a step of 2^-8 relative, over 2h), the slope's own, and h^2 / 6 times the third
    # derivative, at most 3
    bound = 2.0 ** -8 * (up[0].double().abs() + down[0].double().abs()) / (2 * h) + 2.0 ** -8 * dz[0].double().abs() + 0.5 * h * h
    assert ((got - dz[0].double()).abs() <= bound * 1.01).all()


def test_bwd_captured_and_streams(f8):
    gen = torch.Generator(device=DEV).manual_seed(47)
    z, dy = (torch.randn((900, 2056), generator=gen, device=DEV).to(BF) for _ in range(2))
    want = f8.f8_act_bwd(dy, z, f8.F8_ACT_GELU)
    dz, db, top = torch.zeros_like(z), torch.zeros_like(z[0]), torch.zeros((), device=DEV)
    ws = torch.empty(f8.f8_act_bwd_workspace_bytes(900, 2056), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        f8.f8_act_bwd(dy, z, f8.F8_ACT_GELU, dz=dz, dbias=db, amax_out=top, ws=ws)
    for _ in range(2):
        dz.zero_(), db.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dz, want[0]) and torch.equal(db, want[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = f8.f8_act_bwd(dy, z, f8.F8_ACT_GELU, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bwd_empty(f8):
    e = torch.zeros((0, 64), dtype=BF, device=DEV)
    dz, db = f8.f8_act_bwd(e, e, f8.F8_ACT_SILU)
    assert dz.shape == (0, 64) and torch.equal(db, torch.zeros_like(db))
    e = torch.zeros((4, 0), dtype=BF, device=DEV)
    assert f8.f8_act_bwd(e, e, f8.F8_ACT_SILU)[1].shape == (0,)


# ---------------------------------------------------------------- past 2^31 elements
def test_past_2_31_elements_odd_rows(f8):
    """Outputs, residual and kept input past 2^31 elements, of rows that no TMA box takes: the last rows are those of a
    call of their own."""
    M, N, K = 16400, 131077, 16
    a, sa, b, sb, bias, _ = _inputs(M, N, K, 81)
    y = torch.empty((M, N), dtype=BF, device=DEV)
    z = torch.empty_like(y)
    gen = torch.Generator(device=DEV).manual_seed(82)
    last = torch.randn((300, N), generator=gen, device=DEV).to(BF)
    y.zero_()
    y[-300:] = last
    f8.f8_gemm_act(a, b, sa, sb, bias=bias, act=f8.F8_ACT_GELU, residual=y, y=y, z=z)   # in place
    assert y.numel() > 1 << 31
    y1, z1 = f8.f8_gemm_act(a[-300:].contiguous(), b, sa, sb, bias=bias, act=f8.F8_ACT_GELU, residual=last, want_z=True)
    assert torch.equal(y[-300:], y1) and torch.equal(z[-300:], z1)
    y0, z0 = f8.f8_gemm_act(a[:300].contiguous(), b, sa, sb, bias=bias, act=f8.F8_ACT_GELU, residual=torch.zeros_like(last),
                            want_z=True)
    assert torch.equal(y[:300], y0) and torch.equal(z[:300], z0)
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("cols", [8200, 8195])
def test_bwd_past_2_31_elements(f8, cols):
    """The gradient's last rows are those of a call of their own, and the bias's is theirs: the others' dy is 0."""
    rows = (1 << 18) + 77
    gen = torch.Generator(device=DEV).manual_seed(83)
    z, dy = torch.empty((rows, cols), dtype=BF, device=DEV), torch.zeros((rows, cols), dtype=BF, device=DEV)
    z.fill_(0.5)
    for t in (z, dy):
        t[-200:] = torch.randn((200, cols), generator=gen, device=DEV).to(BF)
    assert z.numel() > 1 << 31
    want, _ = f8.f8_act_bwd(dy[-200:].clone(), z[-200:].clone(), f8.F8_ACT_GELU)
    _, _, _, bound = ref.act_bwd(dy[-200:], z[-200:], "gelu")
    exact = ref.act_bwd(dy[-200:], z[-200:], "gelu")[1]
    dz, db = f8.f8_act_bwd(dy, z, f8.F8_ACT_GELU, dz=dy, bias_dtype=torch.float32)
    assert torch.equal(dz[-200:], want) and not dz[:-200].any()
    check(db, exact, bound + rounding(exact, torch.float32), "dbias")
    assert f8.f8_last_device_status() == 0


def test_few_rows_repeat(f8):
    """A decoding step's outputs are the same bits every time, whatever calls run between and whatever the output's memory
    held: sums in rank order, nothing kept from one call for the next."""
    shapes = [(8, 1792, 4096), (8, 4096, 1792), (1, 1024, 4096), (130, 512, 2048)]
    calls = []
    for i, (M, N, K) in enumerate(shapes):
        a, sa, b, sb, bias, res = _inputs(M, N, K, 90 + i)
        y, z = torch.empty_like(res), torch.empty_like(res)
        calls.append(lambda a=a, sa=sa, b=b, sb=sb, bias=bias, res=res, y=y, z=z: f8.f8_gemm_act(
            a, b, sa, sb, bias=bias, act=f8.F8_ACT_SILU, residual=res, y=y, z=z))
    first = []
    for call in calls:
        first.append([t.clone() for t in call()])
        torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(97)
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in torch.randint(0, len(calls), (600,), generator=gen).tolist():
        for t, want in zip(calls[i](), first[i]):
            wrong += (t != want).any()
            t.fill_(float("nan"))
    assert wrong.item() == 0 and f8.f8_last_device_status() == 0
