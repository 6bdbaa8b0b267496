"""The norm over many rows, so that every group of threads takes several and
the slots that bulk copies fill are used again and again, each at the other
phase than before: whole and odd widths of every group size, against the
definition in 64 bits."""
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


SHAPES = [(9001, 96), (9001, 130), (12000, 520), (12001, 777), (9000, 1000), (9001, 1023), (9000, 1500),
          (7000, 2048), (6001, 2051), (6000, 3001), (4001, 4095), (6000, 4096), (3001, 5003), (3000, 5000),
          (2500, 8192), (2501, 8191), (1500, 9000), (1501, 9001), (700, 16400)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", [0, 1], ids=["layer", "rms"])
def test_many_rows(f8, shape, dtype, kind):
    rows, cols = shape
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x = (torch.randn((rows, cols), generator=g, device=DEV) * 1.7 + 0.3).to(dtype)
    w = 1 + 0.3 * torch.randn((cols,), generator=g, device=DEV)
    b = 0.5 * torch.randn((cols,), generator=g, device=DEV)
    dy = (0.02 * torch.randn((rows, cols), generator=g, device=DEV)).to(dtype)
    rms = kind == f8.F8_RMS_NORM
    y, mean, rstd = f8.f8_norm_fwd(x, w, b, kind=kind, eps=EPS)
    ry, rm, rr, by, bm, br = ref.norm_fwd(x, w, b, rms, EPS)
    what = f"{shape} {dtype} kind {kind}"
    ref.check(y, ry, by + ref.rounding(ry, dtype), what + " y")
    ref.check(rstd, rr, br, what + " rstd")
    if not rms:
        ref.check(mean, rm, bm, what + " mean")
    del ry, by
    dx, dw, db = f8.f8_norm_bwd(dy, x, w, mean, rstd, kind=kind, want_db=True)
    rx, rw, rb, bx, bw, bb = ref.norm_bwd(dy, x, w, mean, rstd, rms)
    ref.check(dx, rx, bx + ref.rounding(rx, dtype), what + " dx")
    ref.check(dw, rw, bw + ref.rounding(rw, w.dtype), what + " dw")
    ref.check(db, rb, bb + ref.rounding(rb, w.dtype), what + " db")
    assert f8.f8_last_device_status() == 0
