"""What stands between the Float8 linears of a block, on torch tensors: the GEMM
with a linear's bias, activation and residual in its epilogue, rotary positions,
and the residual stream's update with the norm in front of the next block.

As in ``ops``, every function has the name of the C entry point of include/f8.h
that it calls and only checks and marshals its arguments.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import binding, ops
from .binding import F8_LAYER_NORM, F8_RMS_NORM, _empty, _zero
from .ops import _DTYPES, _call, _dtype

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8


def _arg(what: str, name: str, t: torch.Tensor | None, dtype, shape: tuple, index: int):
    """ops._ptr for a call whose first tensor is on device `index`.  These calls take
    up to ten tensors while a decoding step's kernel runs for a few microseconds, so
    what holds is found in one expression and what does not by ops._ptr."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    return ops._ptr(what, name, t, dtype, shape, torch.device("cuda", index) if index >= 0 else torch.device("cpu"))


def _one(what: str, name: str, t: torch.Tensor | None, index: int):
    """The pointer of one fp32 value (None if not given)."""
    if t is None:
        return None
    if t.dtype is not _F32 or t.numel() != 1:
        raise TypeError(f"{what}: {name} must be one float32 value")
    if t.get_device() != index:
        raise ValueError(f"{what}: tensors on different devices")
    return t.data_ptr()


def _typed(what: str, name: str, t: torch.Tensor | None, shape: tuple, index: int):
    """The pointer and type of a bf16 or fp32 tensor (None and bf16 if not given)."""
    if t is None:
        return 0, binding.F8_BF16
    return _arg(what, name, t, t.dtype, shape, index), _dtype(what, t)


@functools.lru_cache(maxsize=1024)
def _ws_bytes(lib, name: str, rows: int, cols: int, index: int) -> int:
    """The workspace's bytes of a call on device `index`: a training step asks for the
    same few sizes again and again."""
    return int(getattr(lib, name)(rows, cols))


def _ws(what: str, ws: torch.Tensor | None, nbytes: int, like: torch.Tensor, stream):
    """The pointer and size of the workspace, which is allocated if none is given."""
    if ws is None:
        if nbytes == 0:
            return None, None, 0
        ws = _empty(nbytes, _U8, like.device, stream)
    n = ws.numel()
    return ws, _arg(what, "ws", ws, _U8, (n,), like.get_device()), n


# ---------------------------------------------------------------- epilogues
def f8_gemm_act(a: torch.Tensor, b: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor,
                bias: torch.Tensor | None = None, act: int = binding.F8_ACT_NONE,
                residual: torch.Tensor | None = None, y: torch.Tensor | None = None,
                z: torch.Tensor | None = None, want_z: bool = False,
                amax_out: torch.Tensor | None = None, fmt_a: int = binding.F8_E4M3,
                fmt_b: int = binding.F8_E4M3, stream=None):
    """(y, z) of the Float8 GEMM with a linear's epilogue: z = A B^T / (scale_a
    scale_b) + bias, y = act(z) + residual, both bf16 [M, N]; z None unless given
    or wanted.  A [M, K] and B [N, K] are uint8 codes, the bias bf16 or fp32."""
    what = "f8_gemm_act"
    binding._need(what, _U8, a, b)
    (M, K), (N, K2), at = a.shape, b.shape, a.get_device()
    if K2 != K:
        raise ValueError(f"{what}: a and b must have the same K")
    shape = (M, N)
    y = _empty(shape, _BF16, a.device, stream) if y is None else y
    if z is None and want_z:
        z = _empty(shape, _BF16, a.device, stream)
    bias_p, bias_t = _typed(what, "bias", bias, (N,), at)
    _call(what, stream, binding._ptr(a), fmt_a, _arg(what, "b", b, _U8, (N, K), at), fmt_b, M, N, K,
          _one(what, "scale_a", scale_a, at), _one(what, "scale_b", scale_b, at), bias_p, bias_t, act,
          _arg(what, "residual", residual, _BF16, shape, at), _arg(what, "y", y, _BF16, shape, at),
          _arg(what, "z", z, _BF16, shape, at), _one(what, "amax_out", amax_out, at))
    return y, z


def f8_act_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return int(binding.lib().f8_act_bwd_workspace_bytes(rows, cols))


def f8_act_bwd(dy: torch.Tensor, z: torch.Tensor | None, act: int, dz: torch.Tensor | None = None,
               dbias: torch.Tensor | None = None, bias_dtype: torch.dtype = torch.bfloat16,
               want_dz: bool = True, want_dbias: bool = True, amax_out: torch.Tensor | None = None,
               ws: torch.Tensor | None = None, stream=None):
    """(dz, dbias) of f8_gemm_act's epilogue for the gradient dy [rows, cols] of y
    and the z it kept: dz = dy act'(z), dbias its column sums, of `bias_dtype`."""
    what = "f8_act_bwd"
    binding._need(what, _BF16, dy)
    rows, cols = shape = dy.shape
    at = dy.get_device()
    dz = _empty(shape, _BF16, dy.device, stream) if dz is None and want_dz else dz
    dbias = _empty(cols, bias_dtype, dy.device, stream) if dbias is None and want_dbias else dbias
    dbias_p, dbias_t = _typed(what, "dbias", dbias, (cols,), at)
    args = (binding._ptr(dy), _arg(what, "z", z, _BF16, shape, at), act, rows, cols,
            _arg(what, "dz", dz, _BF16, shape, at), dbias_p, dbias_t, _one(what, "amax_out", amax_out, at))
    need = 0
    if ws is None and dbias is not None:
        need = _ws_bytes(binding.lib(), "f8_act_bwd_workspace_bytes", rows, cols, at)
    ws, *space = _ws(what, ws, need, dy, stream)
    _call(what, stream, *args, *space)
    return dz, dbias


# ---------------------------------------------------------------- rotary positions
# the C structs as bytes: built in one step each
_ROPE_ONE, _ROPE_TWO = struct.Struct("=2Q7q"), struct.Struct("=2Q7q2Q7q")
_NORM = struct.Struct("=5i4x3q2f5Q")
_GRADS = struct.Struct("=7Q")


def _heads(what: str, name: str, t: torch.Tensor, out: torch.Tensor, lead: tuple, dim: int, dtype, index: int):
    """The C struct's values of a tensor [*lead, heads, dim] and its output; what does
    not hold is found by name."""
    shape, x, o = t.shape, t.stride(), out.stride()
    if (shape == out.shape and shape[:-2] == lead and shape[-1] == dim and (x[-1] == o[-1] == 1 or dim <= 1)
            and t.dtype is dtype and out.dtype is dtype and t.get_device() == index and out.get_device() == index):
        if len(x) == 4:
            return t.data_ptr(), out.data_ptr(), shape[2], *x[:3], *o[:3]
        return t.data_ptr(), out.data_ptr(), shape[1], 0, *x[:2], 0, *o[:2]
    for n, v in ((name, t), (name + "_out", out)):
        if v.dtype is not dtype:
            raise TypeError(f"{what}: {n} must be {str(dtype).replace('torch.', '')}")
        if v.get_device() != index:
            raise ValueError(f"{what}: tensors on different devices")
        if v.shape[:-2] != lead or v.shape[-1:] != (dim,) or v.dim() != len(lead) + 2:
            raise ValueError(f"{what}: q, k and the outputs must agree in all but the heads")
        if v.stride(-1) != 1 and dim > 1:
            raise ValueError(f"{what}: the columns of {n} must be contiguous")
    raise ValueError(f"{what}: {name}_out must have the shape of {name}")


def f8_rope(q: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
            k: torch.Tensor | None = None, layout: int = binding.F8_ROPE_HALF, scale: float = 1.0,
            inverse: bool = False, q_out: torch.Tensor | None = None,
            k_out: torch.Tensor | None = None, stream=None):
    """(q_out, k_out): the heads' first 2 len(freqs) columns turned by positions *
    freqs.  q and k are bf16 or fp32 [tokens, heads, dim] or [batch, seq, heads,
    dim], of any strides with dense columns; positions int64 [tokens], [batch, seq]
    or [seq], negative where a row is padding; freqs fp64, radians a position
    (f8_rope_frequencies).  q_out may be q, and k_out k.  `inverse` turns back: the
    gradient of the call."""
    what = "f8_rope"
    kind, dtype, at, shape = _dtype(what, q), q.dtype, q.get_device(), q.shape
    if not ops._on_device(q):
        raise ValueError("libf8 takes device tensors only")
    lead, n = shape[:-2], len(shape)
    if n != 4 and n != 3:
        raise ValueError(f"{what}: q must be [tokens, heads, dim] or [batch, seq, heads, dim]")
    batch, seq, dim = lead[0] if n == 4 else 1, lead[-1], shape[-1]
    q_out = _empty(shape, dtype, q.device, stream) if q_out is None else q_out
    first = _heads(what, "q", q, q_out, lead, dim, dtype, at)
    if k is None:
        count, k_out, tensors = 1, None, _ROPE_ONE.pack(*first)
    else:
        k_out = _empty(k.shape, dtype, k.device, stream) if k_out is None else k_out
        count, tensors = 2, _ROPE_TWO.pack(*first, *_heads(what, "k", k, k_out, lead, dim, dtype, at))
    place, steps = positions.shape, positions.stride()
    if place == lead:
        pb, ps = steps if n == 4 else (0, steps[0])
    elif len(place) == 1 and place[0] == seq:
        pb, ps = 0, steps[0]
    else:
        raise ValueError(f"{what}: positions must have q's leading shape, or be [seq]")
    if positions.dtype is not torch.int64:
        raise TypeError(f"{what}: positions must be int64")
    if freqs.dtype is not torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise TypeError(f"{what}: freqs must be a contiguous 1-D float64 tensor")
    if positions.get_device() != at or freqs.get_device() != at:
        raise ValueError(f"{what}: tensors on different devices")
    _call(what, stream, tensors, count, kind, batch, seq, dim, 2 * freqs.shape[0], layout,
          positions.data_ptr(), pb, ps, freqs.data_ptr(), scale, 1 if inverse else 0)
    return q_out, k_out


def f8_rope_frequencies(rot: int, base: float = 10000.0, scaling: int = binding.F8_ROPE_PLAIN,
                        factor: float = 1.0, original: float = 0.0, slow: float = 1.0,
                        fast: float = 32.0, device=None) -> torch.Tensor:
    """freqs of f8_rope [rot / 2] for heads with `rot` turned columns: base^(-2 i /
    rot), changed for a context `factor` times the `original` one as `scaling` says."""
    host = (ctypes.c_double * max(int(rot) // 2, 1))()
    binding._check(binding.lib().f8_rope_frequencies(int(rot), float(base), int(scaling), float(factor),
                                                     float(original), float(slow), float(fast), host),
                   "f8_rope_frequencies")
    return torch.tensor(list(host), dtype=torch.float64, device=device)


# ---------------------------------------------------------------- residual stream
def _residual_norm(what: str, a, r, w_pre, b_pre, w_post, b_post, gate, gate_rows, scale, kind, eps):
    """The C struct of the call, as bytes; a's and r's shapes are the caller's to check."""
    if a.dim() != 2:
        raise TypeError(f"{what} takes 2-D tensors")
    rows, cols = a.shape
    at, shape, wt = a.get_device(), (cols,), w_pre.dtype
    gt, gp = binding.F8_BF16, 0
    if gate is not None:
        gate_rows = max(rows, 1) if gate_rows is None else min(int(gate_rows), 1 << 62)
        if gate_rows < 1:
            raise ValueError(f"{what}: gate_rows must be at least 1")
        whole = gate.dim() == 1 and rows <= gate_rows  # one gate for all rows
        # no rows are those of any number of gates
        groups = gate.shape[0] if rows == 0 and gate.dim() == 2 else -(-rows // gate_rows)
        gp, gt = _typed(what, "gate", gate, shape if whole else (groups, cols), at)
    try:
        types = _DTYPES[a.dtype], _DTYPES[r.dtype], _DTYPES[wt]
    except KeyError:
        raise TypeError(f"{what} takes bfloat16 or float32 tensors") from None
    return _NORM.pack(kind, *types, gt, rows, cols, gate_rows or 1, eps, scale,
                      _arg(what, "w_pre", w_pre, wt, shape, at), _arg(what, "b_pre", b_pre, wt, shape, at),
                      _arg(what, "w_post", w_post, wt, shape, at), _arg(what, "b_post", b_post, wt, shape, at), gp)


def f8_residual_norm_fwd(a: torch.Tensor, r: torch.Tensor, w_pre: torch.Tensor,
                         b_pre: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                         b_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                         gate_rows: int | None = None, scale: float = 1.0, kind: int = F8_RMS_NORM,
                         eps: float = 1e-5, r_out: torch.Tensor | None = None,
                         y: torch.Tensor | None = None, stats: torch.Tensor | None = None,
                         amax_out: torch.Tensor | None = None, stream=None):
    """(r_out, y, stats) of the residual stream r [rows, cols] and a block's output
    a: r_out = scale r + gate norm(a; w_post, b_post) and y = norm(r_out; w_pre,
    b_pre), the next block's input.  Without w_post a is not normed.  gate [ceil(rows
    / gate_rows), cols], one row for each gate_rows rows (default: one, or [cols], for
    all; any number for no rows).  r may be fp32 beside a bf16 a.  stats fp32 [4, rows]
    is the backward's."""
    what = "f8_residual_norm_fwd"
    n = _residual_norm(what, a, r, w_pre, b_pre, w_post, b_post, gate, gate_rows, scale, kind, eps)
    shape, at, xt, rt = a.shape, a.get_device(), a.dtype, r.dtype
    r_out = _empty(shape, rt, a.device, stream) if r_out is None else r_out
    y = _empty(shape, xt, a.device, stream) if y is None else y
    stats = _empty((4, shape[0]), _F32, a.device, stream) if stats is None else stats
    _call(what, stream, n, binding._ptr(a), _arg(what, "r", r, rt, shape, at),
          _arg(what, "r_out", r_out, rt, shape, at), _arg(what, "y", y, xt, shape, at),
          _arg(what, "stats", stats, _F32, (4, shape[0]), at), _one(what, "amax_out", amax_out, at))
    return r_out, y, stats


# the gradients formed by default: (layer norm, w_post given, gate given)
_WANT = {(layer, post, gated): frozenset(
    ["da", "dr", "dw_pre"] + ["db_pre"] * layer + ["dw_post"] * post + ["db_post"] * (layer and post) + ["dgate"] * gated)
    for layer in (False, True) for post in (False, True) for gated in (False, True)}


def f8_residual_norm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return int(binding.lib().f8_residual_norm_bwd_workspace_bytes(rows, cols))


def f8_residual_norm_bwd(dy: torch.Tensor, dr_out: torch.Tensor | None, a: torch.Tensor,
                         r_out: torch.Tensor, w_pre: torch.Tensor, stats: torch.Tensor,
                         w_post: torch.Tensor | None = None, b_post: torch.Tensor | None = None,
                         gate: torch.Tensor | None = None, gate_rows: int | None = None,
                         scale: float = 1.0, kind: int = F8_RMS_NORM, da: torch.Tensor | None = None,
                         dr: torch.Tensor | None = None, dw_pre: torch.Tensor | None = None,
                         db_pre: torch.Tensor | None = None, dw_post: torch.Tensor | None = None,
                         db_post: torch.Tensor | None = None, dgate: torch.Tensor | None = None,
                         want=None, ws: torch.Tensor | None = None, stream=None):
    """(da, dr, dw_pre, db_pre, dw_post, db_post, dgate) of f8_residual_norm_fwd for
    the gradients dy of y and dr_out of r_out (None: zero), from the forward's a,
    r_out and stats.  Formed are the gradients whose buffers are given and those that
    `want` names (by default those of a, r and of what is given, with the biases' for
    F8_LAYER_NORM); the others are None."""
    what = "f8_residual_norm_bwd"
    n = _residual_norm(what, a, r_out, w_pre, None, w_post, b_post, gate, gate_rows, scale, kind, 0.0)
    shape, at, xt, rt, wt = a.shape, a.get_device(), a.dtype, r_out.dtype, w_pre.dtype
    cols = shape[1:]
    if want is None:
        want = _WANT[kind == F8_LAYER_NORM, w_post is not None, gate is not None]
    if want:
        gd, gs = (wt, cols) if gate is None else (gate.dtype, gate.shape)
        new = lambda size, dtype: _empty(size, dtype, a.device, stream)  # noqa: E731
        da = new(shape, xt) if da is None and "da" in want else da
        dr = new(shape, rt) if dr is None and "dr" in want else dr
        dw_pre = new(cols, wt) if dw_pre is None and "dw_pre" in want else dw_pre
        db_pre = new(cols, wt) if db_pre is None and "db_pre" in want else db_pre
        dw_post = new(cols, wt) if dw_post is None and "dw_post" in want else dw_post
        db_post = new(cols, wt) if db_post is None and "db_post" in want else db_post
        dgate = new(gs, gd) if dgate is None and "dgate" in want else dgate
    grads = _GRADS.pack(
        _arg(what, "da", da, xt, shape, at), _arg(what, "dr", dr, rt, shape, at),
        _arg(what, "dw_pre", dw_pre, wt, cols, at), _arg(what, "db_pre", db_pre, wt, cols, at),
        _arg(what, "dw_post", dw_post, wt, cols, at), _arg(what, "db_post", db_post, wt, cols, at),
        0 if dgate is None else _arg(what, "dgate", dgate, wt if gate is None else gate.dtype,
                                     cols if gate is None else gate.shape, at))
    need = 0 if ws is not None else _ws_bytes(binding.lib(), "f8_residual_norm_bwd_workspace_bytes", *shape, at)
    ws, *space = _ws(what, ws, need, a, stream)
    _call(what, stream, n, _arg(what, "dy", dy, xt, shape, at),
          _arg(what, "dr_out", dr_out, rt, shape, at), binding._ptr(a), _arg(what, "r_out", r_out, rt, shape, at),
          _arg(what, "stats", stats, _F32, (4, shape[0]), at), grads, *space)
    if shape[0] == 0 and dgate is not None:
        _zero(dgate, stream)  # a sum over no rows, of as many gates as are given: the C call knows of none
    return da, dr, dw_pre, db_pre, dw_post, db_post, dgate
