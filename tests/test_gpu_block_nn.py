"""Float8LinearAct, ResidualNorm and RotaryPositions on the GPU: under autograd
they give exactly the outputs and gradients of the calls that they wrap, for
leading dimensions, partial and broadcast gradients, pieces of larger buffers;
linears with a bias swapped in a model; and a block made of them, with the q, k, v
group, against the chain of the separate calls, eager and as a CUDA graph."""
import pytest
import torch

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


@pytest.fixture(scope="module")
def f8nn(f8):
    from float8_mixed_precision_gb300 import nn
    return nn


def _rnd(shape, std, seed, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _linear_chain(f8, x, w, b, res, act, dy, grad_format=0):
    """The module's outputs and gradients by the calls."""
    (xq, xt, sx, ax), (wq, wt, sw, aw) = f8.f8_quantize_multi([x, w])
    y, z = f8.f8_gemm_act(xq, wq, sx, sw, bias=b, act=act, residual=res, want_z=True)
    dz, db = f8.f8_act_bwd(dy, z, act, bias_dtype=BF if b is None else b.dtype)
    saved = f8.LinearSaved(xt, wt, torch.stack([ax, sx, aw, sw]))
    dx, dw = f8.f8_linear_bwd(dz, saved, dy_fmt=grad_format)
    return y, dx, dw, db


@pytest.mark.parametrize("act", ["none", "relu2", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("bias", [None, BF, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_linear_act(f8, f8nn, act, bias, residual):
    m = f8nn.Float8LinearAct(160, 272, bias=False, activation=act, device=DEV,
                             b=None if bias is None else torch.nn.Parameter(_rnd(272, 0.3, 1, bias)))
    x, dy = _rnd((4, 24, 160), 1.0, 2).requires_grad_(True), _rnd((4, 24, 272), 0.02, 3)
    r = _rnd((4, 24, 272), 1.0, 4).requires_grad_(True) if residual else None
    y = m(x, r)
    y.backward(dy)
    want = _linear_chain(f8, x.detach().reshape(96, 160), m.weight.detach(), None if bias is None else m.bias.detach(),
                         None if r is None else r.detach().reshape(96, 272), f8nn._ACTIVATIONS[act], dy.reshape(96, 272))
    assert torch.equal(y.reshape(96, 272), want[0]) and torch.equal(x.grad.reshape(96, 160), want[1])
    assert torch.equal(m.weight.grad, want[2])
    if bias is not None:
        assert torch.equal(m.bias.grad, want[3])
    if residual:
        assert torch.equal(r.grad, dy)
    assert f8.f8_last_device_status() == 0


def test_linear_act_partial_gradients(f8, f8nn):
    """Frozen parts give no gradient and change none of the others; broadcast gradients and pieces of buffers are taken."""
    m = f8nn.Float8LinearAct(64, 80, activation="silu", device=DEV)
    flat = _rnd(32 * 64 + 3, 1.0, 5)
    x = flat[3:].reshape(32, 64).detach().requires_grad_(True)
    m(x).float().sum().backward()
    full = x.grad.clone(), m.weight.grad.clone(), m.bias.grad.clone()
    for frozen in ("weight", "bias"):
        m.zero_grad()
        x.grad = None
        getattr(m, frozen).requires_grad_(False)
        m(x).float().sum().backward()
        assert torch.equal(x.grad, full[0]) and getattr(m, frozen).grad is None
        getattr(m, frozen).requires_grad_(True)
    m.zero_grad()
    m(x.detach()).float().sum().backward()
    assert torch.equal(m.weight.grad, full[1]) and torch.equal(m.bias.grad, full[2])
    y = m(x, residual=_rnd((32, 80), 1.0, 6))
    y.float().sum().backward(retain_graph=True)
    y.float().sum().backward()                     # a second pass over the kept graph
    with torch.no_grad():
        assert not m(x).requires_grad


def test_swapped_linears(f8, f8nn):
    net = torch.nn.Sequential(torch.nn.Linear(64, 96), torch.nn.SiLU(), torch.nn.Linear(96, 64, bias=False)).to(DEV, BF)
    w, b = net[0].weight, net[0].bias
    f8nn.to_float8_linears(net)
    assert isinstance(net[0], torch.nn.Linear) and isinstance(net[2], f8nn.Float8Linear)
    f8nn.to_float8_linears(net, biases=True)
    assert isinstance(net[0], f8nn.Float8LinearAct) and net[0].weight is w and net[0].bias is b
    x = _rnd((48, 64), 1.0, 7)
    net(x).float().sum().backward()
    assert w.grad is not None and b.grad is not None and torch.isfinite(w.grad).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "one", "batch", "rows"])
@pytest.mark.parametrize("types", [(BF, BF), (BF, torch.float32)], ids=["bf16", "f32-stream"])
def test_residual_norm(f8, f8nn, kind, post, gate, types):
    shape, dim = (3, 10, 72), 72
    m = f8nn.ResidualNorm(dim, kind=kind, post=post, scale=0.7, device=DEV)
    with torch.no_grad():
        for i, p in enumerate(m.parameters()):
            p.copy_(_rnd(dim, 0.4, 11 + i) + 1)
    a, r = _rnd(shape, 1.5, 21, types[0]).requires_grad_(True), _rnd(shape, 2.0, 22, types[1]).requires_grad_(True)
    g = {None: None, "one": _rnd(dim, 1.0, 23), "batch": _rnd((3, 1, dim), 1.0, 23), "rows": _rnd(shape, 1.0, 23)}[gate]
    g = None if g is None else g.requires_grad_(True)
    r_out, y = m(a, r, g)
    assert r_out.shape == r.shape and r_out.dtype == r.dtype and y.dtype == a.dtype
    dr, dy = _rnd(shape, 0.1, 24, types[1]), _rnd(shape, 0.1, 25, types[0])
    torch.autograd.backward([r_out, y], [dr, dy])
    flat = lambda t: None if t is None else t.detach().reshape(-1, dim)  # noqa: E731
    kw = dict(w_post=None if not post else m.post_weight.detach(),
              b_post=None if m.post_bias is None else m.post_bias.detach(), gate=flat(g),
              gate_rows={None: None, "one": 30, "batch": 10, "rows": 1}[gate], scale=0.7,
              kind=f8.F8_LAYER_NORM if kind == "layer" else f8.F8_RMS_NORM)
    want = f8.f8_residual_norm_fwd(flat(a), flat(r), m.weight.detach(), b_pre=None if m.bias is None else m.bias.detach(), **kw)
    grads = f8.f8_residual_norm_bwd(flat(dy), flat(dr), flat(a), want[0], m.weight.detach(), want[2], **kw)
    assert torch.equal(flat(r_out), want[0]) and torch.equal(flat(y), want[1])
    for t, ref in zip((a, r, m.weight, m.bias, m.post_weight, m.post_bias, g), grads):
        assert (t is None) == (ref is None)
        if t is not None:
            assert torch.equal(t.grad.reshape(ref.shape), ref)
    # one upstream gradient missing
    for out in (r_out, y):
        a.grad = r.grad = None
        r2, y2 = m(a, r, g)
        (r2 if out is r_out else y2).float().sum().backward()
        assert torch.isfinite(a.grad).all() and torch.isfinite(r.grad).all()
    assert f8.f8_last_device_status() == 0


def test_residual_norm_frozen(f8, f8nn):
    m = f8nn.ResidualNorm(64, device=DEV)
    a, r = _rnd((8, 64), 1.0, 31).requires_grad_(True), _rnd((8, 64), 1.0, 32)
    for p in m.parameters():
        p.requires_grad_(False)
    r_out, y = m(a, r)
    (r_out.float().sum() + y.float().sum()).backward()
    assert a.grad is not None and all(p.grad is None for p in m.parameters()) and r.grad is None


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=4.0),
                                     dict(scaling="by_parts", factor=4.0, original=4096.0)])
def test_rotary(f8, f8nn, layout, scaling):
    m = f8nn.RotaryPositions(48, base=5000.0, layout=layout, scale=1.1, **scaling).to(DEV).bfloat16()
    packed = _rnd((2, 9, 8, 64), 1.0, 41).requires_grad_(True)
    pos = torch.arange(9, device=DEV) + 100
    q, k = m(packed[:, :, :6], pos, packed[:, :, 6:])
    dq, dk = _rnd(q.shape, 0.1, 42), _rnd(k.shape, 0.1, 43)
    torch.autograd.backward([q, k], [dq, dk.transpose(2, 3).contiguous().transpose(2, 3)])
    freqs = m.frequencies(DEV)
    assert freqs.dtype == torch.float64
    kw = dict(layout=m.layout, scale=1.1)
    want = f8.f8_rope(packed.detach()[:, :, :6], pos, freqs, k=packed.detach()[:, :, 6:], **kw)
    back = f8.f8_rope(dq, pos, freqs, k=dk, inverse=True, **kw)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(packed.grad[:, :, :6], back[0]) and torch.equal(packed.grad[:, :, 6:], back[1])
    alone = m(packed.detach()[:, :, :6], pos)
    assert torch.equal(alone, want[0])
    packed.grad = None
    q, k = m(packed[:, :, :6], pos, packed[:, :, 6:])
    k.backward(dk)                                  # one of the two alone
    assert torch.equal(packed.grad[:, :, 6:], back[1]) and not packed.grad[:, :, :6].any()


def test_module_refusals(f8nn):
    m = f8nn.Float8LinearAct(64, 64, device=DEV)
    x = _rnd((16, 64), 1.0, 51)
    bad = [(TypeError, lambda: m(x.float())), (ValueError, lambda: m(x[:, :48])), (ValueError, lambda: m(x[:15])),
           (ValueError, lambda: m(x, residual=x[:8])), (TypeError, lambda: m(x, residual=x.float())),
           (ValueError, lambda: f8nn.Float8LinearAct(64, 72)), (ValueError, lambda: f8nn.Float8LinearAct(64, 64, activation="tanh")),
           (ValueError, lambda: f8nn.ResidualNorm(64, kind="batch")), (ValueError, lambda: f8nn.RotaryPositions(64, layout="x")),
           (ValueError, lambda: f8nn.RotaryPositions(64, scaling="x"))]
    n = f8nn.ResidualNorm(64, device=DEV)
    bad += [(ValueError, lambda: n(x, x[:8])), (ValueError, lambda: n(x, x, _rnd((3, 64), 1.0, 52))),
            (ValueError, lambda: n(x, x, _rnd((4, 32), 1.0, 53)))]
    for err, call in bad:
        with pytest.raises(err):
            call()


# ---------------------------------------------------------------- a block
class _Block(torch.nn.Module):
    """A transformer block with norms before and after its parts: q, k and v as one group, rotary positions, attention
    in torch, and the linears with their biases, activation and residual."""

    def __init__(self, f8nn, dim, heads, kv_heads, hidden):
        super().__init__()
        self.heads, self.kv, self.hd = heads, kv_heads, dim // heads
        self.qkv = f8nn.Float8LinearGroup(dim, [dim, self.kv * self.hd, self.kv * self.hd], device=DEV)
        self.rope = f8nn.RotaryPositions(self.hd, layout="half")
        self.out = f8nn.Float8LinearAct(dim, dim, device=DEV)
        self.mid = f8nn.ResidualNorm(dim, device=DEV)
        self.up = f8nn.Float8LinearAct(dim, hidden, activation="gelu_tanh", device=DEV)
        self.down = f8nn.Float8LinearAct(hidden, dim, device=DEV)
        self.end = f8nn.ResidualNorm(dim, device=DEV)

    def attend(self, q, k, v):
        b, s = q.shape[:2]
        rep = self.heads // self.kv
        k, v = k.repeat_interleave(rep, 2), v.repeat_interleave(rep, 2)
        p = torch.einsum("bqhd,bkhd->bhqk", q.float(), k.float()) / self.hd ** 0.5
        p = torch.softmax(p + torch.full((s, s), float("-inf"), device=DEV).triu(1), -1)
        return torch.einsum("bhqk,bkhd->bqhd", p, v.float()).to(BF).reshape(b, s, -1)

    def forward(self, x, stream, gate, positions):
        b, s = x.shape[:2]
        q, k, v = self.qkv(x)
        q, k = self.rope(q.view(b, s, self.heads, self.hd), positions, k.view(b, s, self.kv, self.hd))
        stream, x = self.mid(self.out(self.attend(q, k, v.view(b, s, self.kv, self.hd))), stream, gate)
        return self.end(self.down(self.up(x)), stream, gate)


def _block_inputs(f8nn):
    m = _Block(f8nn, 256, 4, 2, 512)
    x, stream = _rnd((2, 48, 256), 1.0, 61).requires_grad_(True), _rnd((2, 48, 256), 1.0, 62).requires_grad_(True)
    gate = _rnd((2, 256), 0.5, 63).requires_grad_(True)
    pos = torch.arange(48, device=DEV)
    up = _rnd((2, 48, 256), 0.05, 64), _rnd((2, 48, 256), 0.05, 65)
    return m, x, stream, gate, pos, up


def test_block_against_fp32(f8, f8nn):
    """The block against the same formulas in fp32: E4M3 rounds each operand's elements by up to 2^-4 relative (2.6 % rms
    for values spread over a binade), so a linear's output is off by some 4 % and five in a row by less than 15 %."""
    m, x, stream, gate, pos, up = _block_inputs(f8nn)
    outs = m(x, stream, gate, pos)
    torch.autograd.backward(list(outs), list(up))
    got = [*outs, x.grad, stream.grad, gate.grad, m.up.weight.grad, m.up.bias.grad, m.mid.weight.grad, m.out.weight.grad]
    P = {n: p.detach().float().requires_grad_(True) for n, p in m.named_parameters()}
    xr, sr, gr = (t.detach().float().requires_grad_(True) for t in (x, stream, gate))
    b, s = 2, 48
    q, k, v = (xr @ P[f"qkv.weights.{i}"].t() for i in range(3))
    t = pos.double()[:, None] * m.rope.frequencies(DEV)
    cos, sin = t.cos().float()[:, None], t.sin().float()[:, None]

    def turn(h):
        h1, h2 = h.chunk(2, -1)
        return torch.cat((h1 * cos - h2 * sin, h2 * cos + h1 * sin), -1)

    def rms(h, w):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-5) * w
    q, k, v = turn(q.view(b, s, 4, 64)), turn(k.view(b, s, 2, 64)), v.view(b, s, 2, 64)
    k, v = k.repeat_interleave(2, 2), v.repeat_interleave(2, 2)
    p = torch.softmax(torch.einsum("bqhd,bkhd->bhqk", q, k) / 8.0 + torch.full((s, s), float("-inf"), device=DEV).triu(1), -1)
    h = torch.einsum("bhqk,bkhd->bqhd", p, v).reshape(b, s, -1) @ P["out.weight"].t() + P["out.bias"]
    sr2 = sr + gr[:, None] * rms(h, P["mid.post_weight"])
    h = rms(sr2, P["mid.weight"])
    h = torch.nn.functional.gelu(h @ P["up.weight"].t() + P["up.bias"], approximate="tanh") @ P["down.weight"].t() + P["down.bias"]
    sr3 = sr2 + gr[:, None] * rms(h, P["end.post_weight"])
    refs = [sr3, rms(sr3, P["end.weight"])]
    torch.autograd.backward(refs, [u.float() for u in up])
    refs += [xr.grad, sr.grad, gr.grad, P["up.weight"].grad, P["up.bias"].grad, P["mid.weight"].grad, P["out.weight"].grad]
    for i, (u, w) in enumerate(zip(got, refs)):
        rel = ((u.float() - w).norm() / w.norm()).item()
        assert rel < 0.15, (i, rel)
    assert f8.f8_last_device_status() == 0


def test_block_captured(f8, f8nn):
    """A captured step of the block gives the eager step's outputs and gradients at every replay."""
    m, x, stream, gate, pos, up = _block_inputs(f8nn)
    leaves = [x, stream, gate, *m.parameters()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            for p in leaves:
                p.grad = None
            outs = m(x, stream, gate, pos)
            torch.autograd.backward(list(outs), list(up))
        want = [t.detach().clone() for t in (*outs, *(p.grad for p in leaves))]
        del outs
    torch.cuda.current_stream().wait_stream(side)
    for p in leaves:
        p.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = m(x, stream, gate, pos)
        torch.autograd.backward(list(outs), list(up))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip((*outs, *(p.grad for p in leaves)), want):
            assert torch.equal(u, v)


def test_rotary_evaluated_then_trained(f8, f8nn):
    """A module that is first used under inference mode gives the gradients of one that is not."""
    q, pos, dq = _rnd((40, 4, 64), 1.0, 71).requires_grad_(True), torch.arange(40, device=DEV), _rnd((40, 4, 64), 0.1, 72)
    grads = []
    for first in (False, True):
        m = f8nn.RotaryPositions(64)
        if first:
            with torch.inference_mode():
                m(q.detach(), pos)
        q.grad = None
        m(q, pos).backward(dq)
        grads.append(q.grad.clone())
    assert torch.equal(grads[0], grads[1])
