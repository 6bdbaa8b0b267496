"""The casts, GEMMs and linears on a stream that is not the current one, with
outputs, saved buffers and workspaces of their own: the current stream has
writes under way to blocks that it has given back, which are not theirs."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
WAIT = 20_000_000        # cycles that the current stream is kept busy: about 10 ms


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


def _rnd(shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _calls(f8):
    M, N, K = 512, 768, 640
    x, w, dy = _rnd((M, K), 1), _rnd((N, K), 2), _rnd((M, N), 3)
    amax = f8.f8_amax(x)
    q, _, sx, _ = f8.f8_quantize(x)
    wq, _, sw, _ = f8.f8_quantize(w)
    _, saved = f8.f8_linear_fwd(x, w)
    _, group = f8.f8_linear_fwd_group(x, [w, w])
    return {
        "amax": lambda s: f8.f8_amax(x, stream=s),
        "cast_transpose": lambda s: f8.f8_cast_transpose(x, amax, stream=s),
        "quantize": lambda s: f8.f8_quantize(x, stream=s),
        "quantize_multi": lambda s: f8.f8_quantize_multi([x, w], stream=s),
        "quantize_swiglu": lambda s: f8.f8_quantize_swiglu(dy, dy, stream=s),
        "gemm": lambda s: f8.f8_gemm(q, wq, sx, sw, stream=s),
        "gemm_grouped": lambda s: f8.f8_gemm_grouped([(q, wq, sx, sw), (wq, q, sw, sx)], stream=s),
        "linear_fwd": lambda s: f8.f8_linear_fwd(x, w, stream=s),
        "linear_bwd": lambda s: f8.f8_linear_bwd(dy, saved, stream=s),
        "linear_fwd_group": lambda s: f8.f8_linear_fwd_group(x, [w, w], stream=s),
        "linear_bwd_group": lambda s: f8.f8_linear_bwd_group([dy, dy], group, K, stream=s),
        "transpose_u8": lambda s: f8.f8_transpose_u8(q, stream=s),
    }


NAMES = ["amax", "cast_transpose", "quantize", "quantize_multi", "quantize_swiglu", "gemm", "gemm_grouped",
         "linear_fwd", "linear_bwd", "linear_fwd_group", "linear_bwd_group", "transpose_u8"]


def _tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    if isinstance(out, (tuple, list)):
        return [t for o in out for t in _tensors(o)]
    if out is None:
        return []
    # saved buffers; a group's members leave the first two of their own scalars unset
    own = out.scalars if out.x_scalars is None else out.scalars[2:]
    return [t for t in (out.x_t, out.w_t, own, out.x_scalars) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_memory_the_current_stream_still_uses(f8, name):
    call = _calls(f8)[name]
    want = [t.clone() for t in _tensors(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of these sizes and of a workspace's, and small ones for the scalars
    sizes = [max(t.numel() * t.element_size(), 1) for t in want]
    used = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes + [16384, 1 << 20, 4 << 20] + [512] * 8]
    torch.cuda._sleep(WAIT)
    for t in used:
        t.fill_(0x41)
    del used, t
    out = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(_tensors(out), want))
    assert f8.f8_last_device_status() == 0
