"""The norms and the logits' functions of float8_mixed_precision_gb300.nn on the
GPU: under autograd they give exactly the outputs and gradients of the calls
they wrap, for leading dimensions, padded heads, gradients that are broadcast or
missing; and the distilled head of example_distill gives exactly the chain of
the separate calls, eager and as a CUDA graph, and learns."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


def _rnd(shape, std, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


@pytest.mark.parametrize("dtype,wtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                         (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("kind", ["layer", "layer_no_bias", "rms"])
def test_norms(f8, kind, dtype, wtype):
    from float8_mixed_precision_gb300 import nn as f8nn
    shape, dim = (3, 5, 72), 72
    m = (f8nn.RMSNorm(dim, device=DEV, dtype=wtype) if kind == "rms" else
         f8nn.LayerNorm(dim, bias=kind == "layer", device=DEV, dtype=wtype))
    with torch.no_grad():
        for p in m.parameters():
            p.copy_(_rnd(dim, 0.5, 1, wtype) + 1)
    x, g = _rnd(shape, 1.5, 2, dtype).requires_grad_(True), _rnd(shape, 0.1, 3, dtype)
    y = m(x)
    assert y.dtype == dtype and y.shape == x.shape
    y.backward(g)
    k = f8.F8_RMS_NORM if kind == "rms" else f8.F8_LAYER_NORM
    x2 = x.detach().reshape(-1, dim)
    y2, mean, rstd = f8.f8_norm_fwd(x2, m.weight.detach(), None if m.bias is None else m.bias.detach(), kind=k)
    dx, dw, db = f8.f8_norm_bwd(g.reshape(-1, dim), x2, m.weight.detach(), mean, rstd, kind=k,
                                want_db=m.bias is not None)
    assert torch.equal(y.reshape(-1, dim), y2) and torch.equal(x.grad.reshape(-1, dim), dx)
    assert torch.equal(m.weight.grad, dw) and (m.bias is None or torch.equal(m.bias.grad, db))
    assert f8.f8_last_device_status() == 0


def test_norm_partial_gradients(f8):
    """A frozen norm gives dx only, an input without gradient the parameters'
    only; a strided input and a broadcast gradient are taken as they come."""
    from float8_mixed_precision_gb300 import nn as f8nn
    m = f8nn.LayerNorm(40, device=DEV)
    x = _rnd((40, 24), 1.0, 4).t().requires_grad_(True)
    m(x).float().sum().backward()
    full, dw = x.grad.clone(), m.weight.grad.clone()
    x.grad = m.weight.grad = m.bias.grad = None
    m(x.detach()).float().sum().backward()
    assert x.grad is None and torch.equal(m.weight.grad, dw)
    m.weight.grad = m.bias.grad = None
    m.requires_grad_(False)
    m(x).float().sum().backward()
    assert torch.equal(x.grad, full) and m.weight.grad is None
    (g,) = torch.autograd.grad(m(x).float().pow(2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()              # no second derivatives


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_token_logprobs(f8, dtype):
    from float8_mixed_precision_gb300 import nn as f8nn
    lead, vocab, width, T = (2, 9), 1001, 1008, 0.7
    z = _rnd((*lead, width), 2.0, 5, dtype).requires_grad_(True)
    tokens = torch.randint(0, vocab, lead, device=DEV)
    tokens[1, 3] = -1
    logp, ent = f8nn.token_logprobs(z, tokens, temperature=T, vocab=vocab)
    flat = z.detach().reshape(-1, width)
    logp2, ent2, lse, _, _ = f8.f8_token_logprobs(flat[:, :vocab], tokens.reshape(-1), temperature=T)
    assert torch.equal(logp.reshape(-1), logp2) and torch.equal(ent.reshape(-1), ent2)
    ones = torch.ones(18, device=DEV)
    # both gradients (broadcast), and each alone
    for outs, a, b in (((logp.sum() + 0.5 * ent.sum()), ones, 0.5 * ones), (logp.sum(), ones, None),
                       (ent.sum(), None, ones)):
        (got,) = torch.autograd.grad(outs, z, retain_graph=True)
        want = f8.f8_token_logprobs_bwd(flat[:, :vocab], tokens.reshape(-1), lse, ent2, a, b,
                                        temperature=T, dlogits=torch.empty_like(flat))
        assert torch.equal(got.reshape(-1, width), want) and not got[..., vocab:].any()
        assert not got[1, 3].any() and got[0, 0].any()
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("tail", [False, True])
def test_distill_loss(f8, tail):
    from float8_mixed_precision_gb300 import nn as f8nn
    lead, vocab, width, k, T = (2, 7), 777, 784, 12, 1.5 if not tail else 1.0
    z = _rnd((*lead, width), 2.0, 6).requires_grad_(True)
    ids = torch.rand((*lead, vocab), device=DEV).argsort(-1)[..., :k].to(torch.int32)
    ids[0, 0, 5:] = -1
    values = torch.log_softmax(_rnd((*lead, k), 1.0, 7, torch.float32), -1) - 0.2
    loss = f8nn.distill_loss(z, ids, values, temperature=T, tail=tail, vocab=vocab)
    assert loss.shape == lead and loss.dtype == torch.float32
    loss.mean().backward()
    flat, ids2, values2 = z.detach().reshape(-1, width), ids.reshape(-1, k), values.reshape(-1, k)
    l2, lse, rest = f8.f8_distill_fwd(flat[:, :vocab], ids2, values2, temperature=T, tail=tail)
    want = f8.f8_distill_bwd(flat[:, :vocab], ids2, values2, lse, rest, torch.full((14,), 1 / 14, device=DEV),
                             temperature=T, tail=tail, dlogits=torch.empty_like(flat))
    assert torch.equal(loss.detach().reshape(-1), l2) and torch.equal(z.grad.reshape(-1, width), want)
    assert f8.f8_last_device_status() == 0


@pytest.mark.parametrize("tail", [False, True])
def test_distilled_head(f8, tail):
    """student_step against the separate calls, bit for bit, and its loss
    against the definition; the same as a CUDA graph."""
    from float8_mixed_precision_gb300 import example_distill as ex
    M, D, vocab, width, k = 256, 128, 1001, 1008, 16
    x, w, gain = _rnd((M, D), 1.0, 8), _rnd((width, D), 0.1, 9), 1 + _rnd(D, 0.2, 10)
    ids, values = ex.teacher_top(x, _rnd((width, D), 0.2, 11), k, vocab)
    dloss = torch.rand(M, device=DEV) / M
    got = ex.student_step(x, gain, w, ids, values, dloss, vocab, tail)
    y, _, rstd = f8.f8_norm_fwd(x, gain, kind=f8.F8_RMS_NORM)
    logits, saved = f8.f8_linear_fwd(y, w)
    loss, d = f8.f8_distill_fwd_bwd(logits[:, :vocab], ids, values, dloss, tail=tail,
                                    dlogits=torch.empty_like(logits))
    dy, dw = f8.f8_linear_bwd(d, saved)
    dx, dgain, _ = f8.f8_norm_bwd(dy, x, gain, None, rstd, kind=f8.F8_RMS_NORM)
    for a, b, what in zip(got, (loss, dx, dgain, dw), ("loss", "dx", "dgain", "dweight")):
        assert torch.equal(a, b), what
    r = ref.distill(logits[:, :vocab], ids, values, 1.0, tail, dloss)
    ref.check(got[0], r["loss"], r["b_loss"], "loss")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ex.student_step(x, gain, w, ids, values, dloss, vocab, tail)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ex.student_step(x, gain, w, ids, values, dloss, vocab, tail)
    for o in out:
        o.fill_(7.0)
    graph.replay()
    for a, b in zip(out, got):
        assert torch.equal(a, b)
    assert f8.f8_last_device_status() == 0


def test_example_learns(f8, capsys):
    from float8_mixed_precision_gb300 import example_distill as ex
    ex.main(["--tokens", "256", "--features", "128", "--vocab", "1000", "--top", "16", "--steps", "5"])
    line = [s for s in capsys.readouterr().out.splitlines() if s.startswith("loss over")][0]
    first, last = (float(v) for v in line.split(":")[1].split("->"))
    assert last < first
