"""The GEMM epilogue, rotary and residual-norm calls without a GPU: the C calls
reject bad arguments on the host before they touch the device, the Python wrappers
check types, shapes, strides and devices and hand the C calls the argument lists
that include/f8.h declares, and the frequencies, which are formed on the host, are
their formulas'."""
import ctypes
import math

import pytest
import torch

from float8_mixed_precision_gb300 import binding, block, ops

INVALID, ALIGN, SHAPE = 1, 2, 3
P = 1 << 40            # an aligned address that is never dereferenced
P8, P2 = P + 8, P + 2


@pytest.fixture(scope="module")
def L():
    from float8_mixed_precision_gb300 import build
    build.build()
    return binding.lib()


def _refuse(fn, ok, cases):
    for at, value, want in cases:
        args = list(ok)
        args[at] = value
        assert fn(*args) == want, (fn.__name__, at, value, fn(*args))


def test_gemm_act_refusals(L):
    #      a fmt b fmt M N K sa sb bias type act residual y z amax stream
    ok = (P, 0, P, 0, 32, 48, 64, P, P, P, 0, 4, P, 2 * P, 3 * P, P, None)
    _refuse(L.f8_gemm_act, ok, [
        (0, None, INVALID), (2, None, INVALID), (1, 2, INVALID), (3, -1, INVALID), (4, -1, INVALID),
        (7, None, INVALID), (8, None, INVALID), (10, 2, INVALID), (11, 6, INVALID), (11, -1, INVALID),
        (13, None, INVALID), (14, 2 * P, INVALID), (14, P, INVALID),   # z is y, z is the residual
        (6, 65, SHAPE), (6, 0, SHAPE), (4, 1 << 31, SHAPE), (0, P8, ALIGN), (2, P8, ALIGN), (9, P8, ALIGN),
        (12, P8, ALIGN), (13, 2 * P + 8, ALIGN), (14, 3 * P + 8, ALIGN), (15, P2, ALIGN), (7, P2, ALIGN)])


def test_act_bwd_refusals(L):
    #      dy z act rows cols dz dbias type amax ws bytes stream
    ok = (P, P, 3, 640, 64, P, P, 0, P, P, 1 << 20, None)
    _refuse(L.f8_act_bwd, ok, [
        (0, None, INVALID), (1, None, INVALID), (2, 6, INVALID), (3, -1, INVALID), (4, -1, INVALID),
        (5, None, INVALID),                                  # an amax needs dz
        (7, 3, INVALID), (9, None, INVALID), (10, 16, INVALID), (4, 1 << 30, SHAPE), (3, 1 << 60, SHAPE),
        (0, P8, ALIGN), (1, P8, ALIGN), (5, P8, ALIGN), (6, P8, ALIGN), (9, P8, ALIGN), (8, P2, ALIGN)])
    assert L.f8_act_bwd_workspace_bytes(0, 64) == 0
    assert L.f8_act_bwd_workspace_bytes(8, 64) == 0          # one chunk of rows: the sums are the result
    assert L.f8_act_bwd_workspace_bytes(8, 65) >= 65 * 4 and L.f8_act_bwd_workspace_bytes(640, 64) >= 20 * 64 * 4


def _rope_args(**kw):
    t = binding._RopeTensor(P, 2 * P, 4, 4096, 512, 128, 4096, 512, 128)
    for k, v in kw.items():
        setattr(t, k, v)
    return (binding._RopeTensor * 1)(t)


def test_rope_refusals(L):
    #      tensors count type batch seq dim rot layout pos pos_batch pos_seq freqs scale inverse stream
    ok = (_rope_args(), 1, 0, 2, 8, 128, 128, 0, P, 8, 1, P, 1.0, 0, None)
    _refuse(L.f8_rope, ok, [
        (0, None, INVALID), (1, 0, INVALID), (1, 3, INVALID), (2, 2, INVALID), (3, -1, INVALID), (4, -1, INVALID),
        (7, 2, INVALID), (8, None, INVALID), (11, None, INVALID), (12, float("nan"), INVALID),
        (12, float("inf"), INVALID), (6, 0, SHAPE), (6, 127, SHAPE), (6, 130, SHAPE), (5, 1025, SHAPE),
        (4, 1 << 40, SHAPE), (8, P + 4, ALIGN), (11, P + 4, ALIGN), (0, _rope_args(x=P + 1), ALIGN),
        (0, _rope_args(out=P + 1), ALIGN), (0, _rope_args(x=None), INVALID), (0, _rope_args(out=None), INVALID),
        (0, _rope_args(heads=-1), INVALID), (0, _rope_args(heads=1 << 13), SHAPE),
        (0, _rope_args(out=P, out_seq=1024), INVALID),      # in place, but elsewhere
        (0, _rope_args(out_head=0), INVALID), (0, _rope_args(out_seq=0), INVALID),
        (0, _rope_args(out_batch=0), INVALID)])             # outputs on one another


def _norm_args(**kw):
    n = dict(kind=0, x_type=0, r_type=0, w_type=0, gate_type=0, rows=8, cols=64, gate_rows=8, eps=1e-5, scale=1.0,
             w_pre=P, b_pre=P, w_post=P, b_post=P, gate=P)
    n.update(kw)
    return ctypes.byref(binding._ResidualNorm(*n.values()))


BAD_NORMS = [(dict(kind=2), INVALID), (dict(x_type=2), INVALID), (dict(r_type=5), INVALID), (dict(w_type=-1), INVALID),
             (dict(gate_type=2), INVALID), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID),
             (dict(gate_rows=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
             (dict(scale=float("inf")), INVALID), (dict(w_pre=None), INVALID), (dict(w_post=None), INVALID),
             (dict(x_type=1, r_type=0), INVALID),             # an fp32 output beside a bf16 stream
             (dict(cols=1 << 30), SHAPE), (dict(rows=1 << 60), SHAPE), (dict(w_pre=P8), ALIGN),
             (dict(b_pre=P8), ALIGN), (dict(w_post=P8), ALIGN), (dict(b_post=P8), ALIGN), (dict(gate=P8), ALIGN)]


def test_residual_norm_refusals(L):
    #      n a r r_out y stats amax stream
    ok = (_norm_args(), P, 2 * P, 3 * P, 4 * P, P, P, None)
    _refuse(L.f8_residual_norm_fwd, ok, [(0, _norm_args(**kw), want) for kw, want in BAD_NORMS] + [
        (0, None, INVALID), (1, None, INVALID), (2, None, INVALID), (3, None, INVALID), (4, None, INVALID),
        (5, None, INVALID), (3, 4 * P, INVALID), (3, P, INVALID), (4, 2 * P, INVALID),
        (0, _norm_args(x_type=1, r_type=1), INVALID),        # an amax needs a bf16 output
        (1, P8, ALIGN), (2, P8, ALIGN), (3, P8, ALIGN), (4, P8, ALIGN), (5, P2, ALIGN), (6, P2, ALIGN)])
    grads = lambda **kw: ctypes.byref(binding._ResidualNormGrads(**kw))  # noqa: E731
    every = dict(da=5 * P, dr=6 * P, dw_pre=P, db_pre=P, dw_post=P, db_post=P, dgate=P)
    #      n dy dr_out a r_out stats grads ws bytes stream
    ok = (_norm_args(), P, 2 * P, 3 * P, 4 * P, P, grads(**every), P, 1 << 30, None)
    _refuse(L.f8_residual_norm_bwd, ok, [(0, _norm_args(**kw), want) for kw, want in BAD_NORMS] + [
        (0, None, INVALID), (1, None, INVALID), (3, None, INVALID), (4, None, INVALID), (5, None, INVALID),
        (6, None, INVALID), (7, None, INVALID), (8, 16, INVALID),
        (0, _norm_args(w_post=None, b_post=None), INVALID), (0, _norm_args(gate=None), INVALID),
        (6, grads(**(every | dict(da=P))), INVALID), (6, grads(**(every | dict(dr=2 * P))), INVALID),
        (6, grads(**(every | dict(da=4 * P))), INVALID), (6, grads(**(every | dict(dr=3 * P))), INVALID),
        (6, grads(**(every | dict(da=5 * P + 8))), ALIGN), (6, grads(**(every | dict(dgate=P8))), ALIGN),
        (1, P8, ALIGN), (2, 2 * P + 8, ALIGN), (3, 3 * P + 8, ALIGN), (4, 4 * P + 8, ALIGN), (5, P2, ALIGN),
        (7, P8, ALIGN)])
    assert L.f8_residual_norm_bwd_workspace_bytes(0, 64) == 0
    assert L.f8_residual_norm_bwd_workspace_bytes(8, 64) >= 6 * 64 * 4


def test_struct_layout():
    """The structs as C lays them out: pointers and 64-bit integers on 8 bytes, 32-bit ones packed."""
    assert ctypes.sizeof(binding._RopeTensor) == 72
    assert ctypes.sizeof(binding._ResidualNorm) == 24 + 24 + 8 + 40
    assert binding._ResidualNorm.rows.offset == 24 and binding._ResidualNorm.w_pre.offset == 56
    assert ctypes.sizeof(binding._ResidualNormGrads) == 56


# ---------------------------------------------------------------- frequencies
def test_frequencies(L):
    f8 = block
    plain = f8.f8_rope_frequencies(96, 10000.0)
    i = torch.arange(48, dtype=torch.float64)
    want = 10000.0 ** (-2 * i / 96)
    assert plain.dtype == torch.float64 and torch.allclose(plain, want, rtol=1e-14, atol=0)
    linear = f8.f8_rope_frequencies(96, 10000.0, binding.F8_ROPE_LINEAR, factor=4.0)
    assert torch.allclose(linear, want / 4, rtol=1e-14, atol=0)
    # the slowest pair is slowed down by the factor, the fastest kept
    based = f8.f8_rope_frequencies(96, 10000.0, binding.F8_ROPE_BASE, factor=4.0)
    assert based[0] == 1.0 and math.isclose(based[-1], want[-1] / 4, rel_tol=1e-12)
    assert (based[1:] < want[1:]).all()
    parts = f8.f8_rope_frequencies(96, 10000.0, binding.F8_ROPE_BY_PARTS, factor=4.0, original=4096.0, slow=1.0,
                                   fast=32.0)
    turns = 4096.0 * want / (2 * math.pi)
    assert torch.equal(parts[turns >= 32.0], plain[turns >= 32.0])
    assert torch.allclose(parts[turns <= 1.0], want[turns <= 1.0] / 4, rtol=1e-14, atol=0)
    keep = ((turns - 1) / 31).clamp(0, 1)
    assert torch.allclose(parts, want * keep + want / 4 * (1 - keep), rtol=1e-13, atol=0)
    assert 0 < ((keep > 0) & (keep < 1)).sum() < 48


@pytest.mark.parametrize("kw, want", [
    (dict(rot=0), SHAPE), (dict(rot=7), SHAPE), (dict(rot=1026), SHAPE), (dict(base=0.0), INVALID),
    (dict(base=float("nan")), INVALID), (dict(scaling=4), INVALID), (dict(scaling=1, factor=0.0), INVALID),
    (dict(scaling=2, rot=2, factor=2.0), SHAPE), (dict(scaling=3, factor=2.0), INVALID),
    (dict(scaling=3, factor=2.0, original=10.0, slow=4.0, fast=4.0), INVALID)])
def test_frequencies_refusals(L, kw, want):
    with pytest.raises(binding.F8Error) as e:
        block.f8_rope_frequencies(**(dict(rot=8) | kw))
    assert e.value.status == want


# ---------------------------------------------------------------- wrappers
class _Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        fn = getattr(self.real, name)

        def call(*args):
            assert len(args) == len(fn.argtypes), (name, len(args), len(fn.argtypes))
            for a, t in zip(args, fn.argtypes):
                t.from_param(a)                       # what ctypes would refuse
            self.calls.append(name)
            return 4096 if fn.restype is ctypes.c_size_t else 0
        return call


@pytest.fixture()
def rec(L, monkeypatch):
    r = _Recorder(L)
    monkeypatch.setattr(binding, "lib", lambda: r)
    monkeypatch.setattr(binding, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(binding, "_stream", lambda s: 0)
    monkeypatch.setattr(ops, "_on_device", lambda t: True)
    return r


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_every_wrapper_marshals(rec):
    one = torch.ones(1)
    y, z = block.f8_gemm_act(_u8(8, 64), _u8(48, 64), one, one)
    assert y.shape == (8, 48) and z is None
    y, z = block.f8_gemm_act(_u8(8, 64), _u8(48, 64), one, one, bias=torch.zeros(48), act=3, residual=y, want_z=True)
    assert z.shape == (8, 48) and z.dtype == torch.bfloat16
    dz, db = block.f8_act_bwd(y, z, 3, bias_dtype=torch.float32)
    assert dz.shape == (8, 48) and db.shape == (48,) and db.dtype == torch.float32
    assert block.f8_act_bwd(y, None, 0, want_dz=False)[0] is None
    assert block.f8_act_bwd(y, z, 3, want_dbias=False)[1] is None
    f, pos = torch.zeros(32, dtype=torch.float64), torch.zeros(8, dtype=torch.int64)
    q, k = block.f8_rope(_bf(8, 4, 64), pos, f)
    assert q.shape == (8, 4, 64) and k is None
    packed = _bf(2, 8, 12, 64)
    q, k = block.f8_rope(packed[:, :, :8], pos, f, k=packed[:, :, 8:10], inverse=True)
    assert q.shape == (2, 8, 8, 64) and k.shape == (2, 8, 2, 64) and q.is_contiguous()
    block.f8_rope(packed[:, :, :8], pos.expand(2, 8), f, q_out=packed[:, :, :8])
    block.f8_rope(packed.transpose(1, 2).contiguous().transpose(1, 2), pos, f)
    block.f8_rope_frequencies(64)
    a, w = _bf(8, 64), _bf(64)
    r_out, y, stats = block.f8_residual_norm_fwd(a, a.float(), w)
    assert r_out.dtype == torch.float32 and y.dtype == torch.bfloat16 and stats.shape == (4, 8)
    block.f8_residual_norm_fwd(a, a, w, w, w, w, gate=w)
    block.f8_residual_norm_fwd(a, a, w, w, w, w, gate=_bf(3, 64), gate_rows=3, scale=0.5)
    g = block.f8_residual_norm_bwd(a, None, a, r_out, w, stats)
    assert [t is not None for t in g] == [True, True, True, False, False, False, False]
    assert g[1].dtype == torch.float32
    g = block.f8_residual_norm_bwd(a, a, a, a, w, stats, w_post=w, gate=_bf(3, 64), gate_rows=3, kind=0)
    assert all(t is not None for t in g) and g[6].shape == (3, 64)
    g = block.f8_residual_norm_bwd(a, a, a, a, w, stats, want=("dr",))
    assert [t is not None for t in g] == [False, True, False, False, False, False, False]
    names = {n for n in binding.EXPORTS if hasattr(block, n)}
    assert len(names) == 8 and names <= set(rec.calls), sorted(names - set(rec.calls))


def test_wrappers_refuse(rec):
    one, u, v = torch.ones(1), _u8(8, 64), _u8(48, 64)
    y, a, w = _bf(8, 48), _bf(8, 64), _bf(64)
    f, pos, q = torch.zeros(32, dtype=torch.float64), torch.zeros(8, dtype=torch.int64), _bf(8, 4, 64)
    st = torch.zeros(4, 8)
    bad = [
        (TypeError, lambda: block.f8_gemm_act(a, v, one, one)),
        (ValueError, lambda: block.f8_gemm_act(u, _u8(48, 32), one, one)),
        (TypeError, lambda: block.f8_gemm_act(u, v, one.double(), one)),
        (TypeError, lambda: block.f8_gemm_act(u, v, one, torch.ones(2))),
        (ValueError, lambda: block.f8_gemm_act(u, v, one, one, bias=_bf(47))),
        (TypeError, lambda: block.f8_gemm_act(u, v, one, one, bias=_bf(48).half())),
        (TypeError, lambda: block.f8_gemm_act(u, v, one, one, residual=y.float())),
        (ValueError, lambda: block.f8_gemm_act(u, v, one, one, residual=a)),
        (ValueError, lambda: block.f8_gemm_act(u, v, one, one, y=_bf(48, 8).t())),
        (TypeError, lambda: block.f8_act_bwd(y.float(), y, 3)),
        (ValueError, lambda: block.f8_act_bwd(y, a, 3)),
        (ValueError, lambda: block.f8_act_bwd(y, y, 3, dbias=_bf(8))),
        (TypeError, lambda: block.f8_rope(q.half(), pos, f)),
        (TypeError, lambda: block.f8_rope(q, pos.int(), f)),
        (TypeError, lambda: block.f8_rope(q, pos, f.float())),
        (ValueError, lambda: block.f8_rope(q, pos[:7], f)),
        (ValueError, lambda: block.f8_rope(q[0], pos, f)),
        (ValueError, lambda: block.f8_rope(q.transpose(1, 2), pos, f)),
        (TypeError, lambda: block.f8_rope(q, pos, f, k=q.float())),
        (ValueError, lambda: block.f8_rope(q, pos, f, k=_bf(7, 4, 64))),
        (ValueError, lambda: block.f8_rope(q, pos, f, k=_bf(8, 4, 32))),
        (ValueError, lambda: block.f8_rope(q, pos, f, q_out=_bf(8, 4, 32))),
        (TypeError, lambda: block.f8_rope(q, pos, f, q_out=q.float())),
        (TypeError, lambda: block.f8_residual_norm_fwd(a.reshape(-1), a, w)),
        (ValueError, lambda: block.f8_residual_norm_fwd(a, _bf(7, 64), w)),
        (TypeError, lambda: block.f8_residual_norm_fwd(a, a, w, w.float())),
        (ValueError, lambda: block.f8_residual_norm_fwd(a, a, _bf(63))),
        (ValueError, lambda: block.f8_residual_norm_fwd(a, a, w, gate=_bf(2, 64), gate_rows=3)),
        (ValueError, lambda: block.f8_residual_norm_fwd(a, a, w, gate=_bf(2, 64), gate_rows=0)),
        (ValueError, lambda: block.f8_residual_norm_fwd(a, a, w, stats=torch.zeros(8, 4))),
        (TypeError, lambda: block.f8_residual_norm_fwd(a, a, w, y=a.float())),
        (ValueError, lambda: block.f8_residual_norm_bwd(a, a, a, a, w, st, dw_pre=_bf(63))),
        (TypeError, lambda: block.f8_residual_norm_bwd(a, a.float(), a, a, w, st)),
        (ValueError, lambda: block.f8_residual_norm_bwd(_bf(8, 63), a, a, a, w, st)),
    ]
    for i, (err, call) in enumerate(bad):
        rec.calls.clear()
        with pytest.raises(err):
            call()
        assert [c for c in rec.calls if not c.endswith("_bytes")] == [], (i, rec.calls)


def test_no_cpu_path(L):
    with pytest.raises(ValueError, match="device tensors"):
        block.f8_gemm_act(_u8(8, 64), _u8(48, 64), torch.ones(1), torch.ones(1))
    with pytest.raises(ValueError, match="device tensors"):
        block.f8_act_bwd(_bf(8, 64), _bf(8, 64), 3)
    with pytest.raises(ValueError, match="device tensors"):
        block.f8_rope(_bf(8, 4, 64), torch.zeros(8, dtype=torch.int64), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="device tensors"):
        block.f8_residual_norm_fwd(_bf(8, 64), _bf(8, 64), _bf(64))


# ---------------------------------------------------------------- no rows
def test_no_rows_one_gate(rec):
    """The gradient of one gate for all rows is 0 where there are none, and not what memory held."""
    none, w, st = _bf(0, 64), _bf(64), torch.zeros(4, 0)
    dgate = torch.full((64,), 7.0, dtype=torch.bfloat16)
    got = block.f8_residual_norm_bwd(none, None, none, none, w, st, w_post=w, gate=w, dgate=dgate)
    assert got[6] is dgate and not dgate.any()
    rows = _bf(4, 64)
    dgate.fill_(7.0)  # with rows it is the C call's
    block.f8_residual_norm_bwd(rows, None, rows, rows, w, torch.zeros(4, 4), w_post=w, gate=w, dgate=dgate)
    assert (dgate == 7.0).all()


@pytest.mark.parametrize("gate", [(64,), (1, 64), (0, 64), (3, 64)])
def test_no_rows_any_gates(rec, gate):
    """A call of no rows takes gates of any number, as it takes none, and its gradients for them are 0."""
    none, w, st, g = _bf(0, 64), _bf(64), torch.zeros(4, 0), _bf(*gate)
    r_out, y, stats = block.f8_residual_norm_fwd(none, none, w, gate=g)
    assert r_out.shape == y.shape == (0, 64) and stats.shape == (4, 0)
    block.f8_residual_norm_fwd(none, none, w, gate=g, gate_rows=2)
    got = block.f8_residual_norm_bwd(none, none, none, none, w, st, gate=g, dgate=torch.full(gate, 7.0).bfloat16())
    assert got[6].shape == gate and not got[6].any()
    with pytest.raises(ValueError):
        block.f8_residual_norm_fwd(none, none, w, gate=_bf(3, 63))
    with pytest.raises(ValueError):
        block.f8_residual_norm_fwd(_bf(2, 64), _bf(2, 64), w, gate=_bf(0, 64), gate_rows=2)


@pytest.mark.parametrize("lead, gate", [((0,), (64,)), ((0,), (0, 64)), ((0, 5), (64,)), ((0, 5), (0, 64)),
                                        ((0, 5), (0, 1, 64)), ((3, 0), (3, 64)), ((3, 0), (3, 0, 64))])
def test_no_rows_through_the_module(rec, lead, gate):
    from float8_mixed_precision_gb300 import nn
    m = nn.ResidualNorm(64, kind="layer")
    a, r, g = (_bf(*s).requires_grad_(True) for s in ((*lead, 64), (*lead, 64), gate))
    r_out, y = m(a, r, g)
    assert r_out.shape == y.shape == (*lead, 64)
    (r_out.sum() + y.sum()).backward()
    for t in (a, r, g):
        assert t.grad.shape == t.shape and not t.grad.any()
    with pytest.raises(ValueError):
        m(_bf(4, 64), _bf(4, 64), _bf(0, 64))


# ---------------------------------------------------------------- evaluation first
def test_rotary_keeps_no_inference_tensor(rec):
    """What a module keeps of a first use under inference mode serves a later one that trains."""
    from float8_mixed_precision_gb300 import nn
    with torch.inference_mode():
        made = nn.RotaryPositions(64)
        assert not made.frequencies("meta").is_inference() and not made._freqs[None].is_inference()
    q, pos = _bf(8, 4, 64).requires_grad_(True), torch.arange(8)
    for m in (nn.RotaryPositions(64), made):
        with torch.inference_mode():
            m(q.detach(), pos)
        m(q, pos).sum().backward()
        assert q.grad.shape == q.shape


# ---------------------------------------------------------------- nothing to rotate
def test_rope_of_nothing(L):
    """Empty tensors have no address, and views of packed rows strides that their outputs lack: no reason to refuse a call
    that does nothing, nor strides that no element goes by.  (Without a GPU the call ends at the device.)"""
    args = lambda t, count, batch, seq: (t, count, 0, batch, seq, 64, 64, 0, P, seq, 1, P, 1.0, 0, None)  # noqa: E731
    packed = dict(x_batch=3840, x_seq=768, x_head=64, out_batch=2560, out_seq=512, out_head=64)
    for batch, seq in ((0, 5), (2, 0), (0, 0)):
        assert L.f8_rope(*args(_rope_args(x=None, out=None, heads=8, **packed), 1, batch, seq)) not in (INVALID, SHAPE, ALIGN)
    two = (binding._RopeTensor * 2)(binding._RopeTensor(None, None, 0, 3840, 768, 64, 0, 0, 0),
                                    binding._RopeTensor(P, 2 * P, 2, 3840, 768, 64, 640, 128, 64))
    if not torch.cuda.is_available():  # the addresses are not to be read
        assert L.f8_rope(*args(two, 2, 2, 5)) not in (INVALID, SHAPE, ALIGN)
        one = _rope_args(out=P, heads=1, x_batch=9, out_batch=8, x_head=5, out_head=0, out_seq=512)
        assert L.f8_rope(*args(one, 1, 1, 5)) not in (INVALID, SHAPE, ALIGN)
        assert L.f8_rope(*args(one, 1, 2, 5)) == INVALID


def test_gradients_in_one_place_are_refused(L):
    """No gradient may lie in the place of an input or of another gradient."""
    grads = lambda **kw: ctypes.byref(binding._ResidualNormGrads(**kw))  # noqa: E731
    n = _norm_args(w_pre=11 * P, b_pre=12 * P, w_post=13 * P, b_post=14 * P, gate=15 * P)
    every = {k: (20 + i) * P for i, k in enumerate(("da", "dr", "dw_pre", "db_pre", "dw_post", "db_post", "dgate"))}
    call = lambda **kw: L.f8_residual_norm_bwd(n, P, 2 * P, 3 * P, 4 * P, 5 * P, grads(**(every | kw)), 6 * P, 1 << 30, None)  # noqa: E731
    inputs = [i * P for i in (1, 2, 3, 4, 5, 11, 12, 13, 14, 15)]
    for i, name in enumerate(every):
        for place in inputs + [v for k, v in every.items() if k != name]:
            assert call(**{name: place}) == INVALID, (name, place // P)
    if not torch.cuda.is_available():  # the addresses are not to be read
        assert call() not in (INVALID, SHAPE, ALIGN)
        assert call(da=None, dr=None, dw_post=None, db_post=None) not in (INVALID, SHAPE, ALIGN)


@pytest.mark.parametrize("lead, gate, ok", [
    ((3, 10), (3, 1), True), ((3, 10), (3, 10), True), ((3, 10), (1, 1), True), ((3, 10), (3,), True), ((3, 10), (), True),
    ((2, 3, 4), (2, 3), True), ((2, 3, 4), (2, 1, 1), True), ((2, 3, 4), (2, 3, 1), True), ((30,), (10,), True),
    ((3, 10), (1, 10), False), ((10, 10), (1, 10), False), ((2, 3, 4), (1, 3, 4), False), ((2, 3, 4), (2, 1, 4), False),
    ((2, 3, 4), (3, 4), False), ((4, 4), (2, 2), False)])
def test_gates_that_broadcast_otherwise_are_refused(rec, lead, gate, ok):
    """Each gate is that of consecutive rows: a gate whose dimensions would stand for other rows (one for each place of
    every sequence, [1, seq, dim]) is refused, not taken as one for each group of rows."""
    from float8_mixed_precision_gb300 import nn
    m, a, g = nn.ResidualNorm(64), _bf(*lead, 64), _bf(*gate, 64)
    if ok:
        m(a, a, g)
    else:
        with pytest.raises(ValueError, match="leading dimensions"):
            m(a, a, g)
    if len(gate) == len(lead) and all(n in (1, k) for n, k in zip(gate, lead)):
        m(a, a, g.expand(*lead, 64))
