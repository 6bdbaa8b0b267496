"""f8_residual_norm_fwd and _bwd against the definitions in 64 bits
(tests/block_reference.py): rows from one column to past the register path, whole
vectors and odd widths, every mix of types, layer and RMS norm, with and without
the norm after the block, biases and gates; gates of one row, a few rows, and all
rows; in place, the amax, rows of equal values, NaN, differences, fixed order,
streams and captured calls."""
import pytest
import torch

import block_reference as ref
from ops_reference import check, rounding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
STATS = ("mean_post", "rstd_post", "mean_pre", "rstd_pre")
GRADS = ("da", "dr", "dw_pre", "db_pre", "dw_post", "db_post", "dgate")


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


def _inputs(rows, cols, xt=BF, rt=BF, wt=BF, gt=BF, post=True, bias=True, gate_rows=None, seed=1, offset=0.3):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(shape, std, mean, dtype):
        return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)

    s = dict(a=rnd((rows, cols), 1.5, offset, xt), r=rnd((rows, cols), 2.0, -offset, rt),
             w_pre=rnd((cols,), 0.3, 1.0, wt), b_pre=rnd((cols,), 0.5, 0.0, wt) if bias else None,
             w_post=rnd((cols,), 0.3, 1.0, wt) if post else None,
             b_post=rnd((cols,), 0.5, 0.0, wt) if bias and post else None, gate=None, gate_rows=gate_rows)
    if gate_rows is not None:
        s["gate"] = rnd((-(-rows // gate_rows), cols), 0.5, 0.8, gt)
    s["dy"] = rnd((rows, cols), 0.02, 0.0, xt)
    s["dr_out"] = rnd((rows, cols), 0.02, 0.0, rt)
    return s


def _kw(f8, s, layer, scale):
    return dict(w_post=s["w_post"], b_post=s["b_post"], gate=s["gate"], gate_rows=s["gate_rows"], scale=scale,
                kind=f8.F8_LAYER_NORM if layer else f8.F8_RMS_NORM)


def _check(f8, s, layer, scale, what, upstream=True, amax=False):
    rows = s["a"].shape[0]
    stats = torch.full((4, rows), -7.0, device=DEV)
    top = torch.full((), -1.0, device=DEV) if amax else None
    r_out, y, _ = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], eps=EPS, stats=stats,
                                          amax_out=top, **_kw(f8, s, layer, scale))
    want = ref.residual_norm_fwd(s["a"], s["r"], s["w_pre"], s["b_pre"], s["w_post"], s["b_post"], s["gate"],
                                 s["gate_rows"], scale, layer, EPS)
    for name, got in (("r_out", r_out), ("y", y)):
        v, b = want[name]
        check(got, v, b + rounding(v, got.dtype), f"{what} {name}")
    for i, name in enumerate(STATS):
        if name not in want or (not layer and name.startswith("mean")):
            assert (stats[i] == -7.0).all(), f"{what} {name} was written"
        else:
            check(stats[i], *want[name], f"{what} {name}")
    if amax:
        assert top.item() == y.float().abs().max().item()
    dr_out = s["dr_out"] if upstream else None
    got = f8.f8_residual_norm_bwd(s["dy"], dr_out, s["a"], r_out, s["w_pre"], stats, want=_all(s),
                                  **_kw(f8, s, layer, scale))
    want = ref.residual_norm_bwd(s["dy"], dr_out, s["a"], r_out, stats, s["w_pre"], s["w_post"], s["b_post"],
                                 s["gate"], s["gate_rows"], scale, layer)
    for name, t in zip(GRADS, got):
        assert (t is not None) == (name in _all(s)), name
        if t is not None:
            v, b = want[name]
            check(t, v.reshape(t.shape), (b + rounding(v, t.dtype)).reshape(t.shape), f"{what} {name}")
    assert f8.f8_last_device_status() == 0
    return r_out, y, stats, got


def _all(s):
    names = {"da", "dr", "dw_pre", "db_pre"}
    if s["w_post"] is not None:
        names |= {"dw_post", "db_post"}
    if s["gate"] is not None:
        names.add("dgate")
    return names


# every path of the width rules, odd ones, one row, one column
SHAPES = [(1, 1), (3, 2), (5, 8), (7, 64), (33, 129), (64, 512), (9, 520), (17, 2047), (40, 2048), (6, 4096),
          (13, 4097), (31, 5003), (5, 8192), (3, 8200), (4, 16384), (2, 16383), (3, 16392), (2, 20001), (700, 1024),
          (1300, 96), (400, 4096)]
TYPES = [(BF, BF, BF), (BF, F32, BF), (F32, F32, F32), (BF, BF, F32), (F32, F32, BF)]


@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(f8, shape, layer):
    for i, (xt, rt, wt) in enumerate(TYPES[:3]):
        s = _inputs(*shape, xt, rt, wt, gt=xt, gate_rows=shape[0], seed=i)
        _check(f8, s, layer, 0.75, f"{shape} {xt} {rt}", amax=xt == BF)


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("post, bias, gate_rows, upstream", [
    (True, True, 5, True), (True, False, None, True), (False, True, 7, False), (False, False, None, False),
    (True, True, 1, False), (False, False, 1, True)])
def test_parts(f8, types, layer, post, bias, gate_rows, upstream):
    for cols in (136, 1048, 2050):
        s = _inputs(37, cols, *types, gt=F32 if gate_rows == 7 else BF, post=post, bias=bias, gate_rows=gate_rows)
        _check(f8, s, layer, -1.5, f"{cols} columns", upstream=upstream)


@pytest.mark.parametrize("rows", [1, 2, 150, 153, 1000])
@pytest.mark.parametrize("gate_rows", [1, 2, 3, 7, 64, 149, 500, 1 << 40])
def test_gates(f8, rows, gate_rows):
    """Gates that change with every row, in the middle of a block's rows, and never."""
    for cols in (520, 1203):
        s = _inputs(rows, cols, gate_rows=min(gate_rows, rows), seed=gate_rows % 100)
        s["gate_rows"] = gate_rows
        _check(f8, s, True, 1.0, f"{rows} rows by {gate_rows}")


@pytest.mark.parametrize("layer, bias", [(True, True), (False, False)], ids=["layer", "rms"])
@pytest.mark.parametrize("cols", [4098, 4104, 4608, 4999, 5113, 5114, 5120, 5128])
def test_wide_blocks(f8, cols, layer, bias):
    """Widths just above a block's usual columns."""
    for i, (rt, rows, gate_rows) in enumerate([(BF, 21, 1), (F32, 200, 67), (BF, 333, 333), (F32, 3, 2)]):
        s = _inputs(rows, cols, BF, rt, gate_rows=gate_rows, bias=bias, seed=i)
        _check(f8, s, layer, 0.75, f"{rows}x{cols} by {gate_rows} {rt}")


@pytest.mark.parametrize("gate_rows", [137, 100, 72, 71, 50, 8])
@pytest.mark.parametrize("rows, cols", [(2500, 4099), (3001, 1003), (2500, 2047), (2500, 2052)])
def test_odd_widths_many_gates(f8, rows, cols, gate_rows):
    """Gates about as long as the rows that units share, longer and shorter; none of the partial rows lies past the
    workspace."""
    s = _inputs(rows, cols, BF, F32, gate_rows=gate_rows, seed=gate_rows)
    r_out, y, stats, want = _check(f8, s, True, 0.75, f"{rows}x{cols} by {gate_rows}")
    n = f8.f8_residual_norm_bwd_workspace_bytes(rows, cols)
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    got = f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], r_out, s["w_pre"], stats, ws=ws[:n], want=_all(s),
                                  **_kw(f8, s, True, 0.75))
    assert (ws[n:] == 0x5A).all()
    for u, v in zip(got, want):
        assert torch.equal(u, v)


@pytest.mark.parametrize("cols", [1000, 1003, 4099, 4104])
def test_frozen_parts(f8, cols):
    """Each gradient alone is the one that comes with all others."""
    s = _inputs(300, cols, gate_rows=40)
    kw = _kw(f8, s, True, 0.75)
    r_out, _, stats, want = _check(f8, s, True, 0.75, f"{cols} columns")
    for i, name in enumerate(GRADS):
        got = f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], r_out, s["w_pre"], stats, want=(name,), **kw)
        assert [j for j, t in enumerate(got) if t is not None] == [i]
        assert torch.equal(got[i], want[i]), name


def test_one_gate_for_all(f8):
    s = _inputs(40, 256, gate_rows=40)
    want = _check(f8, s, False, 1.0, "rows")
    s["gate"], s["gate_rows"] = s["gate"][0], None
    got = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], eps=EPS, **_kw(f8, s, False, 1.0))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], got[0], s["w_pre"], got[2], **_kw(f8, s, False, 1.0))
    assert g[6].shape == (256,) and torch.equal(g[6], want[3][6][0])


@pytest.mark.parametrize("cols", [264, 1001, 4096, 18000])
@pytest.mark.parametrize("rt", [BF, F32])
def test_in_place(f8, cols, rt):
    s = _inputs(90, cols, BF, rt, gate_rows=30)
    kw = dict(b_pre=s["b_pre"], eps=EPS, **_kw(f8, s, True, 0.5))
    r_out, y, _ = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], **kw)
    a, r = s["a"].clone(), s["r"].clone()
    f8.f8_residual_norm_fwd(a, r, s["w_pre"], r_out=r, y=a, **kw)
    assert torch.equal(r, r_out) and torch.equal(a, y)


@pytest.mark.parametrize("cols", [96, 1000, 4096])
def test_flat_rows(f8, cols):
    """Rows of one value: the deviation is eps alone; and rows of zeros."""
    s = _inputs(6, cols, F32, F32, F32)
    s["a"][0], s["a"][1], s["r"][1], s["a"][2], s["r"][2] = 3.0, 0.0, 0.0, 1e4, -1e4
    r_out, y, stats = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], eps=EPS,
                                              **_kw(f8, s, True, 1.0))
    for t in (r_out, y, stats):
        assert torch.isfinite(t).all()
    # a flat row's differences to its mean are the mean's rounding alone
    assert (r_out[0] - s["r"][0] - s["b_post"]).abs().max() <= 64 * 2.0 ** -24 * 3.0 / EPS ** 0.5 * 2.5 + 1e-5
    g = f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], r_out, s["w_pre"], stats, **_kw(f8, s, True, 1.0))
    assert all(t is None or torch.isfinite(t).all() for t in g)


@pytest.mark.parametrize("cols", [264, 1001, 4096])
def test_nan_stays_in_its_row(f8, cols):
    s = _inputs(50, cols, gate_rows=10)
    kw = _kw(f8, s, True, 1.0)
    want = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], eps=EPS, **kw)
    s["a"][17, 3] = float("nan")
    s["r"][29, 5] = float("inf")
    top = torch.zeros((), device=DEV)
    got = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], eps=EPS, amax_out=top, **kw)
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_NONFINITE
    clean = torch.ones(50, dtype=torch.bool, device=DEV)
    clean[17] = clean[29] = False
    for u, v in zip(got[:2], want[:2]):
        assert torch.equal(u[clean], v[clean])
    assert torch.isnan(got[1][17]).all() and torch.isnan(got[1][29]).any()


@pytest.mark.parametrize("cols", [9, 131, 1001, 4095, 5003])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rt", [BF, F32], ids=["bf16", "f32"])
def test_neighbours_of_odd_rows(f8, cols, kind, rt):
    """Rows that share their first and last 16 bytes with others: NaN and infinities at a row's ends stay there, forward
    and backward, and rows behind it are as without them."""
    layer = kind == "layer"
    s = _inputs(40, cols, BF, rt, gate_rows=40)
    kw = _kw(f8, s, layer, 1.0)
    want = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], eps=EPS, **kw)
    names = ("da", "dr")
    grads = f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], want[0], s["w_pre"], want[2], want=names, **kw)[:2]
    bad = [3, 11, 26]
    dirty = dict(s, a=s["a"].clone(), r=s["r"].clone(), dy=s["dy"].clone(), dr_out=s["dr_out"].clone())
    for name in ("a", "r", "dy", "dr_out"):
        dirty[name][3, -1], dirty[name][11, 0], dirty[name][26, -1] = float("nan"), float("inf"), float("-inf")
    got = f8.f8_residual_norm_fwd(dirty["a"], dirty["r"], s["w_pre"], b_pre=s["b_pre"], eps=EPS, **kw)
    clean = torch.ones(40, dtype=torch.bool, device=DEV)
    clean[bad] = False
    for u, v in zip(got[:2], want[:2]):
        assert torch.equal(u[clean], v[clean])
    back = f8.f8_residual_norm_bwd(dirty["dy"], dirty["dr_out"], dirty["a"], got[0], s["w_pre"], got[2], want=names, **kw)[:2]
    for u, v in zip(back, grads):
        assert torch.equal(u[clean], v[clean])
    f8.f8_last_device_status()


def test_differences(f8):
    """The gradients against differences of the forward call along random directions, in fp32."""
    s = _inputs(24, 200, F32, F32, F32, gt=F32, gate_rows=5, seed=3)
    kw = _kw(f8, s, True, 0.8)
    names = ("a", "r", "w_pre", "b_pre", "w_post", "b_post", "gate")

    def value(t):
        r_out, y, _ = f8.f8_residual_norm_fwd(t["a"], t["r"], t["w_pre"], b_pre=t["b_pre"], eps=EPS,
                                              **(kw | {k: t[k] for k in ("w_post", "b_post", "gate")}))
        return (r_out.double() * s["dr_out"].double()).sum() + (y.double() * s["dy"].double()).sum()

    r_out, _, stats = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], eps=EPS, **kw)
    grads = f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], r_out, s["w_pre"], stats, want=_all(s), **kw)
    h = 2.0 ** -6
    for name, g in zip(names, grads):
        d = torch.randn(s[name].shape, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
        up, down = value(s | {name: s[name] + h * d}), value(s | {name: s[name] - h * d})
        along = (g.double() * d.double()).sum()
        # 9600 terms of some 0.02 with fp32 errors of up to 2^-19, over 2h; and h^2 times the third derivative, which
        # for rows of deviation 1 and random directions stays below the first-order terms' size
        size = (g.double().abs() * d.double().abs()).sum()
        assert ((up - down) / (2 * h) - along).abs() <= 9600 * 0.02 * 2.0 ** -19 / h + 4 * h * h * size, name


@pytest.mark.parametrize("cols", [520, 4096, 5003])
def test_same_bits_again(f8, cols):
    s = _inputs(1500, cols, gate_rows=400)
    first = _check(f8, s, True, 1.0, "first")
    kw = _kw(f8, s, True, 1.0)
    again = f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], first[0], s["w_pre"], first[2], want=_all(s), **kw)
    for u, v in zip(again, first[3]):
        assert torch.equal(u, v)
    # one gradient alone is the same
    for i, name in enumerate(GRADS):
        alone = f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], first[0], s["w_pre"], first[2], want=(name,), **kw)
        assert torch.equal(alone[i], first[3][i]) and sum(t is not None for t in alone) == 1


def test_empty(f8):
    z = torch.zeros((0, 64), dtype=BF, device=DEV)
    w = torch.ones(64, dtype=BF, device=DEV)
    top = torch.full((), 5.0, device=DEV)
    r_out, y, stats = f8.f8_residual_norm_fwd(z, z, w, w_post=w, amax_out=top)
    assert y.shape == (0, 64) and top.item() == 0
    g = f8.f8_residual_norm_bwd(z, None, z, z, w, stats, w_post=w)
    assert not g[2].any() and not g[4].any()


def test_captured_and_streams(f8):
    s = _inputs(300, 2056, gate_rows=77)
    kw = _kw(f8, s, True, 1.0)
    fwd = lambda **k: f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], eps=EPS, **kw, **k)  # noqa: E731
    want = fwd()
    bwd = lambda **k: f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], want[0], s["w_pre"], want[2],  # noqa: E731
                                              want=_all(s), **kw, **k)
    grads = bwd()
    out = [torch.zeros_like(t) for t in want]
    gout = {n: torch.zeros_like(t) for n, t in zip(GRADS, grads)}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fwd(r_out=out[0], y=out[1], stats=out[2])
        bwd(**gout)
    for _ in range(2):
        for t in [*out, *gout.values()]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want))
        assert all(torch.equal(u, v) for u, v in zip(gout.values(), grads))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, ggot = fwd(stream=side), bwd(stream=side)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want)) and all(torch.equal(u, v) for u, v in zip(ggot, grads))


def test_ready_for_the_cast(f8):
    """The amax of the producing pass quantises y as f8_quantize does."""
    s = _inputs(256, 512)
    top = torch.zeros((), device=DEV)
    _, y, _ = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], amax_out=top)
    q, qt, scale = f8.f8_cast_transpose(y, top)
    q2, qt2, scale2, amax2 = f8.f8_quantize(y)
    assert torch.equal(q, q2) and torch.equal(qt, qt2) and scale.item() == scale2.item()


def test_past_2_31_elements(f8):
    """Rows whose elements lie past 2^31: the last one is that of a call of its own."""
    rows, cols = (1 << 19) + 3, 4100
    a = torch.zeros((rows, cols), dtype=BF, device=DEV)
    r = torch.zeros((rows, cols), dtype=BF, device=DEV)
    s = _inputs(1, cols, gate_rows=1)
    a[-1], r[-1] = s["a"][0], s["r"][0]
    kw = _kw(f8, s, True, 1.0) | {"gate_rows": rows}
    want = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], **kw)
    got = f8.f8_residual_norm_fwd(a, r, s["w_pre"], b_pre=s["b_pre"], r_out=r, y=a, **kw)
    assert a.numel() > 1 << 31 and torch.equal(got[0][-1:], want[0]) and torch.equal(got[1][-1:], want[1])


@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("cols, rt", [(4100, F32), (4099, BF), (4097, F32), (16391, BF)])
def test_past_2_31_elements_both_passes(f8, cols, rt, layer):
    """Rows of both passes past 2^31 elements, odd widths and those past the register path among them: the last rows are
    the definition's, and as the gradients of the others are 0, so are the sums.  (The order in which a row of an odd width
    is summed goes by where it starts in the tensor's vectors, so a call of these rows alone may differ in a last bit.)"""
    rows, some = (1 << 31) // cols + 77, 50
    s = _inputs(some, cols, BF, rt, gate_rows=some, seed=cols)
    kw = _kw(f8, s, layer, 0.75)

    def long(t, fill):
        v = torch.full((rows, cols), fill, dtype=t.dtype, device=DEV)
        v[-some:] = t
        return v
    a, r = long(s["a"], 0.25), long(s["r"], -1.0)
    assert a.numel() > 1 << 31
    one = kw | {"gate_rows": rows}
    y = torch.empty_like(a)
    r_out, y, stats = f8.f8_residual_norm_fwd(a, r, s["w_pre"], b_pre=s["b_pre"], eps=EPS, r_out=r, y=y, **one)
    want = ref.residual_norm_fwd(s["a"], s["r"], s["w_pre"], s["b_pre"], s["w_post"], s["b_post"], s["gate"], some, 0.75,
                                 layer, EPS)
    for name, got in (("r_out", r_out), ("y", y)):
        v, b = want[name]
        check(got[-some:], v, b + rounding(v, got.dtype), name)
    for i, name in enumerate(STATS):
        if layer or not name.startswith("mean"):
            check(stats[i, -some:], *want[name], name)
    dy, dr_out = long(s["dy"], 0.0), long(s["dr_out"], 0.0)
    grads = f8.f8_residual_norm_bwd(dy, dr_out, a, r_out, s["w_pre"], stats, want=_all(s), da=y, **one)
    want = ref.residual_norm_bwd(s["dy"], s["dr_out"], s["a"], r_out[-some:], stats[:, -some:], s["w_pre"], s["w_post"],
                                 s["b_post"], s["gate"], some, 0.75, layer)
    for name, got in zip(GRADS, grads):
        v, b = want[name]
        if name in ("da", "dr"):
            assert not got[:-some].any(), name
            got = got[-some:]
        check(got, v.reshape(got.shape), (b + rounding(v, got.dtype)).reshape(got.shape), name)
    assert f8.f8_last_device_status() == 0
