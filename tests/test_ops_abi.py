"""The norm, log-probability and distillation calls without a GPU: the C calls
reject bad arguments on the host before they touch the device, and the Python
wrappers check types, shapes, strides and devices and hand the C calls the
argument lists that include/f8.h declares."""
import ctypes

import pytest
import torch

from float8_mixed_precision_gb300 import binding, ops

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


def test_norm_refusals(L):
    #      x  type w  b  type kind rows cols eps y mean rstd amax stream
    ok = (P, 0, P, P, 0, 0, 4, 64, 1e-5, P, P, P, P, None)
    _refuse(L.f8_norm_fwd, ok, [
        (0, None, INVALID), (2, None, INVALID), (9, None, INVALID), (1, 2, INVALID), (4, 7, INVALID),
        (5, 2, INVALID), (6, -1, INVALID), (7, -64, INVALID), (8, -1.0, INVALID),
        (8, float("nan"), INVALID), (1, 1, INVALID),          # an amax needs a bf16 output
        (0, P8, ALIGN), (2, P8, ALIGN), (3, P8, ALIGN), (9, P8, ALIGN), (10, P2, ALIGN),
        (11, P2, ALIGN), (12, P2, ALIGN), (7, 1 << 31, SHAPE), (6, 1 << 60, SHAPE)])
    #      dy x type w type mean rstd kind rows cols dx dw db ws bytes stream
    ok = (P, P, 0, P, 0, P, P, 0, 4, 64, P, P, P, P, 1 << 30, None)
    _refuse(L.f8_norm_bwd, ok, [
        (0, None, INVALID), (1, None, INVALID), (3, None, INVALID), (5, None, INVALID),
        (6, None, INVALID), (13, None, INVALID), (14, 16, INVALID), (2, -1, INVALID), (7, 9, INVALID),
        (0, P8, ALIGN), (1, P8, ALIGN), (10, P8, ALIGN), (11, P8, ALIGN), (12, P8, ALIGN),
        (13, P8, ALIGN), (6, P2, ALIGN)])
    #      x w b type kind rows cols eps y mean rstd amax scale q q_t ws bytes stream
    ok = (P, P, P, 0, 0, 16, 64, 1e-5, P, P, P, P, P, P, P, P, 1 << 20, None)
    _refuse(L.f8_quantize_norm, ok, [
        (0, None, INVALID), (1, None, INVALID), (8, None, INVALID), (11, None, INVALID),
        (15, None, INVALID), (16, 100, INVALID), (13, P8, ALIGN), (14, P8, ALIGN), (12, P2, ALIGN)])
    assert L.f8_norm_bwd_workspace_bytes(0, 64) == 0
    assert L.f8_norm_bwd_workspace_bytes(8, 64) >= 2 * 64 * 4


def test_logprob_refusals(L):
    #      logits type rows vocab ld tokens T k logp ent lse ids top stream
    ok = (P, 0, 4, 100, 104, P, 1.0, 5, P, P, P, P, P, None)
    _refuse(L.f8_token_logprobs, ok, [
        (0, None, INVALID), (1, 2, INVALID), (2, -1, INVALID), (3, 0, INVALID), (4, 99, INVALID),
        (5, None, INVALID), (6, 0.0, INVALID), (6, -1.0, INVALID), (6, float("inf"), INVALID),
        (6, 1e-40, INVALID), (7, -1, INVALID), (7, 101, SHAPE), (11, None, INVALID),
        (12, None, INVALID), (0, P8, ALIGN), (5, P + 4, ALIGN), (8, P2, ALIGN), (9, P2, ALIGN),
        (10, P2, ALIGN), (11, P2, ALIGN), (12, P2, ALIGN), (2, 1 << 40, SHAPE)])
    big = list(ok)
    big[3] = big[4] = (1 << 22) + 1
    assert L.f8_token_logprobs(*big) == SHAPE
    big[3] = big[4] = 4096
    big[7] = 257
    assert L.f8_token_logprobs(*big) == SHAPE
    #      logits type rows vocab ld tokens lse ent dlogp dent T dlogits ldd amax stream
    ok = (P, 0, 4, 100, 104, P, P, P, P, P, 1.0, 2 * P, 104, P, None)
    _refuse(L.f8_token_logprobs_bwd, ok, [
        (0, None, INVALID), (6, None, INVALID), (7, None, INVALID), (5, None, INVALID),
        (11, None, INVALID), (12, 99, INVALID), (1, 1, INVALID), (10, 0.0, INVALID),
        (11, 2 * P + 8, ALIGN), (13, P2, ALIGN), (6, P2, ALIGN)])
    args = list(ok)
    args[11], args[12] = P, 108          # the logits' own buffer with other rows
    assert L.f8_token_logprobs_bwd(*args) == INVALID


def test_distill_refusals(L):
    #      logits type rows vocab ld ids values k T tail loss lse rest stream
    ok = (P, 0, 4, 100, 104, P, P, 8, 1.0, 1, P, P, P, None)
    _refuse(L.f8_distill_fwd, ok, [
        (0, None, INVALID), (5, None, INVALID), (6, None, INVALID), (7, 0, INVALID), (7, 257, SHAPE),
        (8, 0.0, INVALID), (9, 2, INVALID), (10, None, INVALID), (11, None, INVALID),
        (12, None, INVALID), (4, 50, INVALID), (5, P2, ALIGN), (6, P2, ALIGN), (10, P2, ALIGN),
        (12, P2, ALIGN), (0, P8, ALIGN)])
    #      logits type rows vocab ld ids values k T tail lse rest dloss dlogits ldd amax stream
    ok = (P, 0, 4, 100, 104, P, P, 8, 1.0, 1, P, P, P, 2 * P, 104, P, None)
    _refuse(L.f8_distill_bwd, ok, [
        (10, None, INVALID), (11, None, INVALID), (12, None, INVALID), (13, None, INVALID),
        (14, 99, INVALID), (1, 1, INVALID), (13, 2 * P + 8, ALIGN), (12, P2, ALIGN), (15, P2, ALIGN)])
    #      logits type rows vocab ld ids values k T tail dloss loss dlogits ldd amax stream
    ok = (P, 0, 4, 100, 104, P, P, 8, 1.0, 0, P, P, 2 * P, 104, P, None)
    _refuse(L.f8_distill_fwd_bwd, ok, [
        (10, None, INVALID), (11, None, INVALID), (12, None, INVALID), (13, 99, INVALID),
        (1, 1, INVALID), (12, 2 * P + 8, ALIGN), (10, P2, ALIGN), (11, P2, ALIGN)])


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


def test_every_wrapper_marshals(rec):
    x, w = _bf(8, 64), _bf(64)
    y, mean, rstd = ops.f8_norm_fwd(x, w, w)
    assert mean.shape == rstd.shape == (8,)
    assert ops.f8_norm_fwd(x.float(), w, kind=binding.F8_RMS_NORM)[1] is None
    dx, dw, db = ops.f8_norm_bwd(x, x, w, mean, rstd)
    assert dx.shape == x.shape and dw.shape == db.shape == w.shape
    assert ops.f8_norm_bwd(x, x, w, None, rstd, kind=binding.F8_RMS_NORM)[2] is None
    assert ops.f8_norm_bwd(x, x, w, mean, rstd, want_dx=False)[0] is None
    ops.f8_quantize_norm(x, w, w)
    z, tok = _bf(8, 100), torch.zeros(8, dtype=torch.int64)
    logp, ent, lse, ids, top = ops.f8_token_logprobs(z, tok, top_k=5)
    assert ids.shape == top.shape == (8, 5) and ids.dtype == torch.int32
    assert ops.f8_token_logprobs(z)[0] is None and ops.f8_token_logprobs(z)[3] is None
    assert ops.f8_token_logprobs_bwd(z, tok, lse, ent, logp, ent).shape == (8, 100)
    v = torch.zeros((8, 5))
    loss, lse, rest = ops.f8_distill_fwd(z, ids, v, tail=True)
    assert rest.shape == (8,) and ops.f8_distill_fwd(z, ids, v)[2] is None
    ops.f8_distill_bwd(z, ids, v, lse, rest, loss, tail=True)
    ops.f8_distill_fwd_bwd(z, ids, v, loss)
    # a view of a padded buffer: its rows lie apart
    wide = _bf(8, 104)
    assert ops._rows("t", "logits", wide[:, :100])[1] == 104
    d = ops.f8_distill_fwd_bwd(wide[:, :100], ids, v, loss, dlogits=wide)[1]
    assert d is wide
    names = {n for n in binding.EXPORTS if hasattr(ops, n)}
    assert names <= set(rec.calls), sorted(names - set(rec.calls))


def test_wrappers_refuse(rec):
    x, w, one = _bf(8, 64), _bf(64), torch.ones(8)
    z, tok = _bf(8, 100), torch.zeros(8, dtype=torch.int64)
    ids, v = torch.zeros((8, 5), dtype=torch.int32), torch.zeros((8, 5))
    bad = [
        (TypeError, lambda: ops.f8_norm_fwd(x.half(), w)),
        (TypeError, lambda: ops.f8_norm_fwd(x.reshape(-1), w)),
        (ValueError, lambda: ops.f8_norm_fwd(x, _bf(63))),
        (TypeError, lambda: ops.f8_norm_fwd(x, w, w.float())),
        (ValueError, lambda: ops.f8_norm_fwd(x, w, y=_bf(8, 63))),
        (TypeError, lambda: ops.f8_norm_fwd(x, w, y=x.float())),
        (TypeError, lambda: ops.f8_norm_fwd(x, w, amax_out=torch.zeros(2))),
        (TypeError, lambda: ops.f8_norm_bwd(x.float(), x, w, one, one)),
        (ValueError, lambda: ops.f8_norm_bwd(x, x, w, one, torch.ones(7))),
        (TypeError, lambda: ops.f8_quantize_norm(x.float(), w)),
        (TypeError, lambda: ops.f8_token_logprobs(z.half(), tok)),
        (TypeError, lambda: ops.f8_token_logprobs(z, tok.int())),
        (ValueError, lambda: ops.f8_token_logprobs(z, tok[:7])),
        (ValueError, lambda: ops.f8_token_logprobs(z.t().contiguous().t(), tok)),
        (ValueError, lambda: ops.f8_token_logprobs(z[:1].expand(8, 100), tok)),
        (TypeError, lambda: ops.f8_token_logprobs_bwd(z, tok, one, one, one, one, dlogits=z.float())),
        (ValueError, lambda: ops.f8_token_logprobs_bwd(z, tok, one, one, one, one, dlogits=_bf(8, 99))),
        (TypeError, lambda: ops.f8_distill_fwd(z, ids.long(), v)),
        (TypeError, lambda: ops.f8_distill_fwd(z, ids, v.bfloat16())),
        (ValueError, lambda: ops.f8_distill_fwd(z, ids, v[:, :4])),
        (TypeError, lambda: ops.f8_distill_fwd(z, ids[0], v[0])),
        (ValueError, lambda: ops.f8_distill_fwd_bwd(z, ids, v, one[:3])),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
        assert rec.calls == [], (i, rec.calls)


def test_no_cpu_path(L):
    with pytest.raises(ValueError, match="device tensors"):
        ops.f8_norm_fwd(_bf(8, 64), _bf(64))
    with pytest.raises(ValueError, match="device tensors"):
        ops.f8_token_logprobs(_bf(8, 64))
    with pytest.raises(ValueError, match="device tensors"):
        ops.f8_distill_fwd(_bf(8, 64), torch.zeros((8, 2), dtype=torch.int32), torch.zeros((8, 2)))
