"""Calls on a stream that is not the current one, with outputs and workspaces
of their own: memory that the current stream still uses, or takes up next, is
not theirs."""
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


def _rnd(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _calls(f8):
    """name: (call of a stream -> outputs, bytes of its workspace)."""
    x, dy, w = _rnd((2000, 2048), 1), _rnd((2000, 2048), 2), _rnd(2048, 3)
    _, mean, rstd = f8.f8_norm_fwd(x, w, w)
    z = _rnd((600, 5003), 4, torch.float32)
    tokens = torch.randint(0, 5003, (600,), device=DEV)
    logp, ent, lse, ids, top = f8.f8_token_logprobs(z, tokens, top_k=8)
    one = torch.ones(600, device=DEV)
    loss, dlse, rest = f8.f8_distill_fwd(z, ids, top, tail=True)
    return {
        "norm_fwd": (lambda s: f8.f8_norm_fwd(x, w, w, stream=s), 0),
        "norm_bwd": (lambda s: f8.f8_norm_bwd(dy, x, w, mean, rstd, stream=s),
                     f8.f8_norm_bwd_workspace_bytes(2000, 2048)),
        "quantize_norm": (lambda s: f8.f8_quantize_norm(x, w, w, stream=s), f8.f8_quantize_workspace_bytes()),
        "token_logprobs": (lambda s: f8.f8_token_logprobs(z, tokens, top_k=8, stream=s), 0),
        "token_logprobs_bwd": (lambda s: f8.f8_token_logprobs_bwd(z, tokens, lse, ent, one, one, stream=s), 0),
        "distill_fwd": (lambda s: f8.f8_distill_fwd(z, ids, top, tail=True, stream=s), 0),
        "distill_bwd": (lambda s: f8.f8_distill_bwd(z, ids, top, dlse, rest, one, tail=True, stream=s), 0),
        "distill_fwd_bwd": (lambda s: f8.f8_distill_fwd_bwd(z, ids, top, one, tail=True, stream=s), 0),
    }


NAMES = ["norm_fwd", "norm_bwd", "quantize_norm", "token_logprobs", "token_logprobs_bwd", "distill_fwd",
         "distill_bwd", "distill_fwd_bwd"]
WAIT = 20_000_000        # cycles that a stream is kept busy: about 10 ms


def _tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_memory_the_current_stream_still_uses(f8, name, handle):
    """The current stream has writes under way to blocks that it has given back."""
    call, ws = _calls(f8)[name]
    want = [t.clone() for t in _tensors(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sizes = [t.numel() * t.element_size() for t in want] + ([ws] if ws else [])
    used = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
    torch.cuda._sleep(WAIT)
    for t in used:
        t.fill_(0x41)
    del used, t
    out = call(side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(_tensors(out), want))
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("name", ["norm_bwd", "quantize_norm"])
def test_memory_the_current_stream_takes_next(f8, name):
    """The call's workspace is not handed to the current stream while the
    call waits on its own."""
    call, ws = _calls(f8)[name]
    want = [t.clone() for t in _tensors(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    out = call(side)
    mine = [torch.empty(ws, dtype=torch.uint8, device=DEV) for _ in range(4)]
    for t in mine:
        t.fill_(0x41)
    torch.cuda.synchronize()
    assert all(int(t.min()) == int(t.max()) == 0x41 for t in mine)
    assert all(torch.equal(a, b) for a, b in zip(_tensors(out), want))
    assert f8.f8_last_device_status() == 0


def test_outputs_can_be_dropped_and_used_here(f8):
    """Outputs belong to the call's stream and to the current one: dropped
    while either uses them, their memory is not taken up by the other."""
    x, w = _rnd((2000, 2048), 1), _rnd(2048, 3)
    want = f8.f8_norm_fwd(x, w, w)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    y, mean, rstd = f8.f8_norm_fwd(x, w, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(WAIT)
    copy = torch.empty_like(want)
    copy.copy_(y)
    n = y.numel() * 2
    del y, mean, rstd
    with torch.cuda.stream(side):
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0x41)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
