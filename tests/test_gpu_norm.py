"""f8_norm_fwd, f8_norm_bwd and f8_quantize_norm against the definition in 64
bits (tests/ops_reference.py) on every kernel path: rows held by a warp or a
block, whole vectors and odd widths, widths past the register path, bf16 and
fp32, layer and RMS norm, with and without a bias; rows of equal values, large
offsets, NaN; statistics, streams, CUDA graphs, in-place calls and refusals."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


def _inputs(rows, cols, dtype, wtype, seed, offset=0.3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn((rows, cols), generator=g, device=DEV) * 1.7 + offset).to(dtype)
    w = (1 + 0.3 * torch.randn((cols,), generator=g, device=DEV)).to(wtype)
    b = (0.5 * torch.randn((cols,), generator=g, device=DEV)).to(wtype)
    dy = (0.02 * torch.randn((rows, cols), generator=g, device=DEV)).to(dtype)
    return x, w, b, dy


# (rows, cols): every path of the width rules, odd ones, one row, one column
SHAPES = [(1, 1), (3, 2), (5, 8), (7, 64), (33, 129), (64, 512), (9, 520), (17, 2047), (40, 2048),
          (6, 4096), (13, 4097), (31, 5003), (5, 8192), (3, 8200), (4, 16384), (2, 16383),
          (3, 16392), (2, 20001), (700, 1024), (1300, 96)]
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
         (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)]


def _check_fwd(f8, x, w, b, kind, what):
    y, mean, rstd = f8.f8_norm_fwd(x, w, b, kind=kind, eps=EPS)
    rms = kind == f8.F8_RMS_NORM
    ry, rm, rr, by, bm, br = ref.norm_fwd(x, w, b, rms, EPS)
    ref.check(y, ry, by + ref.rounding(ry, x.dtype), what + " y")
    ref.check(rstd, rr, br, what + " rstd")
    if rms:
        assert mean is None
    else:
        ref.check(mean, rm, bm, what + " mean")
    return mean, rstd


def _check_bwd(f8, dy, x, w, mean, rstd, kind, what):
    rms = kind == f8.F8_RMS_NORM
    dx, dw, db = f8.f8_norm_bwd(dy, x, w, mean, rstd, kind=kind, want_db=True)
    rx, rw, rb, bx, bw, bb = ref.norm_bwd(dy, x, w, mean, rstd, rms)
    ref.check(dx, rx, bx + ref.rounding(rx, x.dtype), what + " dx")
    ref.check(dw, rw, bw + ref.rounding(rw, w.dtype), what + " dw")
    ref.check(db, rb, bb + ref.rounding(rb, w.dtype), what + " db")
    return dx, dw, db


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", [0, 1], ids=["layer", "rms"])
def test_against_definition(f8, shape, kind):
    for i, (dt, wt) in enumerate(TYPES):
        x, w, b, dy = _inputs(*shape, dt, wt, seed=100 * i + shape[0] + shape[1])
        what = f"{shape} {dt} {wt} kind {kind}"
        mean, rstd = _check_fwd(f8, x, w, b, kind, what)
        _check_fwd(f8, x, w, None, kind, what + " no bias")
        _check_bwd(f8, dy, x, w, mean, rstd, kind, what)
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("cols", [256, 4096, 4099, 16400])
def test_parts_of_the_backward(f8, cols):
    x, w, b, dy = _inputs(50, cols, torch.bfloat16, torch.bfloat16, 7)
    _, mean, rstd = f8.f8_norm_fwd(x, w, b)
    dx, dw, db = f8.f8_norm_bwd(dy, x, w, mean, rstd)
    only = f8.f8_norm_bwd(dy, x, w, mean, rstd, want_dw=False, want_db=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
    only = f8.f8_norm_bwd(dy, x, w, mean, rstd, want_dx=False)
    assert only[0] is None and torch.equal(only[1], dw) and torch.equal(only[2], db)
    only = f8.f8_norm_bwd(dy, x, w, mean, rstd, want_dx=False, want_dw=False)
    assert torch.equal(only[2], db)
    # the sums over rows have one order
    again = f8.f8_norm_bwd(dy, x, w, mean, rstd)
    assert all(torch.equal(a, c) for a, c in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("cols", [512, 4096, 5001, 16400])
def test_in_place(f8, cols):
    x, w, b, dy = _inputs(20, cols, torch.bfloat16, torch.bfloat16, 8)
    y, mean, rstd = f8.f8_norm_fwd(x, w, b)
    dx, dw, db = f8.f8_norm_bwd(dy, x, w, mean, rstd)
    x2 = x.clone()
    f8.f8_norm_fwd(x2, w, b, y=x2)
    assert torch.equal(x2, y)
    for alias in ("dy", "x"):
        x2, dy2 = x.clone(), dy.clone()
        got = f8.f8_norm_bwd(dy2, x2, w, mean, rstd, dx=dy2 if alias == "dy" else x2)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_hard_rows(f8, dt):
    cols = 1024
    x, w, b, _ = _inputs(8, cols, dt, torch.float32, 9)
    x[0] = 0.0
    x[1] = 3.0                       # no variance: y = b, rstd = 1/sqrt(eps)
    x[2] = 1000.0 + x[2].float()     # an offset of hundreds of deviations
    x[3] = x[3] * 1e-4               # a variance far below eps
    x[4] = x[4] * 1e15
    for kind in (0, 1):
        _check_fwd(f8, x, w, b, kind, f"hard rows kind {kind}")
    x[5, 17] = float("nan")
    x[6, 1] = float("inf")
    y, mean, rstd = f8.f8_norm_fwd(x, w, b)
    bad = torch.isnan(y).any(1).cpu().tolist()
    assert bad == [False] * 5 + [True, True, False]
    assert f8.f8_last_device_status() == 0          # only the amax looks for non-finite values


def test_gradient_against_differences(f8):
    """Central differences of the 64-bit forward's scalar sum(y dy)."""
    x, w, b, dy = _inputs(3, 40, torch.float32, torch.float32, 11)
    for kind in (0, 1):
        _, mean, rstd = f8.f8_norm_fwd(x, w, b, kind=kind)
        dx, dw, db = f8.f8_norm_bwd(dy, x, w, mean, rstd, kind=kind, want_db=True)

        def scalar(xx, ww, bb):
            return (ref.norm_fwd(xx, ww, bb, kind == 1, EPS)[0] * dy.double()).sum()

        for t, grad in ((0, dx), (1, dw), (2, db)):
            args = [x.double(), w.double(), b.double()]
            num = torch.zeros_like(args[t])
            flat = args[t].reshape(-1)
            h = 1e-5
            for i in range(flat.numel()):
                keep = flat[i].item()
                flat[i] = keep + h
                up = scalar(*args)
                flat[i] = keep - h
                num.reshape(-1)[i] = (up - scalar(*args)) / (2 * h)
                flat[i] = keep
            # differences: h^2 times third derivatives of order 1, and 1e-16 / h
            assert (grad.double() - num).abs().max().item() <= 1e-7


@pytest.mark.parametrize("shape", [(16, 64), (128, 4096), (40, 1000), (3, 5001), (2, 16640)], ids=str)
def test_quantize_norm(f8, shape):
    """Equal to f8_norm_fwd followed by f8_quantize, bit for bit."""
    x, w, b, _ = _inputs(*shape, torch.bfloat16, torch.bfloat16, 12)
    for kind in (0, 1):
        amax = torch.empty((), dtype=torch.float32, device=DEV)
        y, mean, rstd = f8.f8_norm_fwd(x, w, b, kind=kind, amax_out=amax)
        assert amax.item() == y.float().abs().max().item()
        q, qt, sc, am = f8.f8_quantize(y)
        got = f8.f8_quantize_norm(x, w, b, kind=kind)
        want = (q, qt, sc, am, y, mean, rstd)
        for g, r in zip(got, want):
            assert (g is None and r is None) or torch.equal(g, r)
    assert f8.f8_last_device_status() == 0
    x[0, 0] = float("inf")
    f8.f8_quantize_norm(x, w, b)
    assert f8.f8_last_device_status() == f8.binding.F8_ERR_NONFINITE


def test_no_rows(f8):
    w = torch.ones(64, device=DEV)
    x = torch.empty((0, 64), device=DEV)
    y, mean, rstd = f8.f8_norm_fwd(x, w)
    assert y.shape == (0, 64)
    dx, dw, db = f8.f8_norm_bwd(x, x, w, mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    assert f8.f8_last_device_status() == 0


def test_streams_and_graph(f8):
    x, w, b, dy = _inputs(300, 2048, torch.bfloat16, torch.bfloat16, 13)
    y, mean, rstd = f8.f8_norm_fwd(x, w, b)
    dx, dw, db = f8.f8_norm_bwd(dy, x, w, mean, rstd)
    out = {n: torch.zeros_like(t) for n, t in (("y", y), ("mean", mean), ("rstd", rstd), ("dx", dx),
                                               ("dw", dw), ("db", db))}
    ws = torch.empty(f8.f8_norm_bwd_workspace_bytes(300, 2048), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        f8.f8_norm_fwd(x, w, b, y=out["y"], mean=out["mean"], rstd=out["rstd"], stream=stream)
        f8.f8_norm_bwd(dy, x, w, out["mean"], out["rstd"], dx=out["dx"], dw=out["dw"], db=out["db"],
                       ws=ws, stream=stream)

    want = dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in out.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in out)
    assert f8.f8_last_device_status() == 0


def test_past_2_31_elements(f8):
    """Offsets past 32 bits: the last rows of a tensor of more than 2^31 elements."""
    cols = 8192
    rows = (1 << 31) // cols + 9
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(14)
    x[-9:] = torch.randn((9, cols), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    y, mean, rstd = f8.f8_norm_fwd(x, w, None, kind=f8.F8_RMS_NORM)
    small = f8.f8_norm_fwd(x[-9:].clone(), w, None, kind=f8.F8_RMS_NORM)
    assert torch.equal(y[-9:], small[0]) and torch.equal(rstd[-9:], small[2])
    assert not y[:-9:4096].any()
    dx, dw, _ = f8.f8_norm_bwd(y, x, w, None, rstd, kind=f8.F8_RMS_NORM)
    sx, sw, _ = f8.f8_norm_bwd(y[-9:].clone(), x[-9:].clone(), w, None, rstd[-9:].clone(),
                               kind=f8.F8_RMS_NORM)
    assert torch.equal(dx[-9:], sx)
    # nine rows of terms, one rounding to bf16 on each side
    assert (dw.float() - sw.float()).abs().max() <= 2 ** -7 * sw.float().abs().max()
    assert f8.f8_last_device_status() == 0
