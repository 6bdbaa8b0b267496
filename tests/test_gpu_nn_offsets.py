"""The norm modules and the logits' functions on tensors that start anywhere in
memory: rows past the first of an odd width, parameters and gradients that are
pieces of larger buffers."""
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


def _rnd(shape, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norms(f8, kind, dtype):
    from float8_mixed_precision_gb300 import nn as f8nn
    dim = 51
    x, g, flat = _rnd((9, dim), 1, dtype), _rnd((9, dim), 2, dtype), _rnd(2 * dim + 1, 3, dtype)
    res = []
    for moved in (False, True):
        m = f8nn.LayerNorm(dim, device=DEV, dtype=dtype) if kind == "layer" else f8nn.RMSNorm(dim, device=DEV, dtype=dtype)
        w, b, xs, gs = flat[1:dim + 1], flat[dim + 1:], x[1:], g[1:]
        if not moved:
            w, b, xs, gs = w.clone(), b.clone(), xs.clone(), gs.clone()
        m.weight = torch.nn.Parameter(w)
        if kind == "layer":
            m.bias = torch.nn.Parameter(b)
        xs = xs.detach().requires_grad_(True)
        assert (xs.data_ptr() % 16 != 0) == moved and (m.weight.data_ptr() % 16 != 0) == moved
        y = m(xs)
        y.backward(gs)
        res.append([y.detach(), xs.grad] + [p.grad for p in m.parameters()])
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_logits(f8, dtype):
    from float8_mixed_precision_gb300 import nn as f8nn
    vocab, k = 1003, 5
    z = _rnd((8, vocab), 4, dtype)
    tokens = torch.randint(0, vocab, (8,), device=DEV)
    ids = torch.rand((8, vocab), device=DEV).argsort(1)[:, :k].to(torch.int32)
    values = torch.log_softmax(_rnd((8, k), 5, torch.float32), 1) - 0.1
    res = []
    for moved in (False, True):
        zs = (z[1:] if moved else z[1:].clone()).detach().requires_grad_(True)
        assert (zs.data_ptr() % 16 != 0) == moved
        logp, ent = f8nn.token_logprobs(zs, tokens[1:])
        loss = f8nn.distill_loss(zs, ids[1:], values[1:], tail=True)
        (a,) = torch.autograd.grad((logp + 0.3 * ent).sum(), zs)
        (b,) = torch.autograd.grad(loss.sum(), zs)
        res.append([logp.detach(), ent.detach(), loss.detach(), a, b])
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert f8.f8_last_device_status() == 0
