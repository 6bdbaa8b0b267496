"""What stands between the Float8 linears of a block, on torch tensors: the GEMM
with a linear's bias, activation and residual in its epilogue, rotary positions,
and the residual stream's update with the norm in front of the next block.

As in ``ops``, every function has the name of the C entry point of include/f8.h
that it calls and only checks and marshals its arguments.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding, ops
from .binding import F8_LAYER_NORM, F8_RMS_NORM, _empty
from .ops import _bytes, _call, _dtype, _ptr, _scalar


# ---------------------------------------------------------------- epilogues
def _bias(what: str, bias: torch.Tensor | None, cols: int, dev):
    """The pointer and type of a bias [cols], bf16 or fp32."""
    if bias is None:
        return None, binding.F8_BF16
    return _ptr(what, "bias", bias, bias.dtype, (cols,), dev), _dtype(what, bias)


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
    binding._need(what, torch.uint8, a, b)
    M, K = a.shape
    N, dev = b.shape[0], a.device
    if b.shape[1] != K:
        raise ValueError(f"{what}: a and b must have the same K")
    y = _empty((M, N), torch.bfloat16, dev, stream) if y is None else y
    if z is None and want_z:
        z = _empty((M, N), torch.bfloat16, dev, stream)
    bf = torch.bfloat16
    _call(what, stream, binding._ptr(a), int(fmt_a), _ptr(what, "b", b, torch.uint8, (N, K), dev),
          int(fmt_b), M, N, K, _scalar(what, scale_a, dev, "scale_a"),
          _scalar(what, scale_b, dev, "scale_b"), *_bias(what, bias, N, dev), int(act),
          _ptr(what, "residual", residual, bf, (M, N), dev), _ptr(what, "y", y, bf, (M, N), dev),
          _ptr(what, "z", z, bf, (M, N), dev), _scalar(what, amax_out, dev))
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
    binding._need(what, torch.bfloat16, dy)
    rows, cols = shape = dy.shape
    dev = dy.device
    dz = _empty(shape, torch.bfloat16, dev, stream) if dz is None and want_dz else dz
    dbias = _empty(cols, bias_dtype, dev, stream) if dbias is None and want_dbias else dbias
    bf = torch.bfloat16
    args = (binding._ptr(dy), _ptr(what, "z", z, bf, shape, dev), int(act), rows, cols,
            _ptr(what, "dz", dz, bf, shape, dev), *_bias(what, dbias, cols, dev),
            _scalar(what, amax_out, dev))
    if ws is None and dbias is not None:
        ws = _empty(max(f8_act_bwd_workspace_bytes(rows, cols), 1), torch.uint8, dev, stream)
    _call(what, stream, *args, *_bytes(what, ws, dev))
    return dz, dbias


# ---------------------------------------------------------------- rotary positions
def _heads(what: str, name: str, t: torch.Tensor, like: torch.Tensor | None = None) -> tuple:
    """(batch, seq, heads, dim) and the strides of the first three, of a tensor
    [tokens, heads, dim] or [batch, seq, heads, dim] with dense columns."""
    if like is not None:
        if t.dtype != like.dtype:
            raise TypeError(f"{what}: {name} must be {str(like.dtype).replace('torch.', '')}")
        if t.device != like.device:
            raise ValueError(f"{what}: tensors on different devices")
        if t.dim() != like.dim():
            raise ValueError(f"{what}: {name} must have as many dimensions as q")
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        shape, stride = (1, *shape), (0, *stride)
    elif len(shape) != 4:
        raise ValueError(f"{what}: {name} must be [tokens, heads, dim] or [batch, seq, heads, dim]")
    if shape[3] > 1 and stride[3] != 1:
        raise ValueError(f"{what}: the columns of {name} must be contiguous")
    return shape, stride


def _rope_tensor(what: str, name: str, x: torch.Tensor, out: torch.Tensor | None, like, stream):
    """The C struct of a tensor and its output, the output, and the shape."""
    shape, sx = _heads(what, name, x, like)
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    elif out.shape != x.shape:
        raise ValueError(f"{what}: {name}_out must have the shape of {name}")
    _, so = _heads(what, name + "_out", out, x)
    return (x.data_ptr(), out.data_ptr(), shape[2], sx[0], sx[1], sx[2], so[0], so[1], so[2]), out, shape


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
    kind = _dtype(what, q)
    if not ops._on_device(q):
        raise ValueError("libf8 takes device tensors only")
    dev = q.device
    first, q_out, (batch, seq, _, dim) = _rope_tensor(what, "q", q, q_out, None, stream)
    if k is None:
        tensors = (binding._RopeTensor * 1)(first)
    else:
        second, k_out, (b2, s2, _, d2) = _rope_tensor(what, "k", k, k_out, q, stream)
        if b2 != batch or s2 != seq or d2 != dim:
            raise ValueError(f"{what}: q and k must agree in all but the heads")
        tensors = (binding._RopeTensor * 2)(first, second)
    if positions.dtype != torch.int64:
        raise TypeError(f"{what}: positions must be int64")
    lead = q.shape[:-2]
    if positions.shape == lead:
        pb, ps = (0, positions.stride(0)) if len(lead) == 1 else positions.stride()
    elif positions.dim() == 1 and positions.shape[0] == seq:
        pb, ps = 0, positions.stride(0)
    else:
        raise ValueError(f"{what}: positions must have q's leading shape, or be [seq]")
    if positions.device != dev or freqs.device != dev:
        raise ValueError(f"{what}: tensors on different devices")
    if freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise TypeError(f"{what}: freqs must be a contiguous 1-D float64 tensor")
    _call(what, stream, tensors, len(tensors), kind, batch, seq, dim, 2 * freqs.shape[0], int(layout),
          positions.data_ptr(), pb, ps, freqs.data_ptr(), float(scale), int(bool(inverse)))
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
    """The C struct of the call; a and r are checked here, b's and w's types too."""
    if a.dim() != 2:
        raise TypeError(f"{what} takes 2-D tensors")
    rows, cols = a.shape
    dev, shape = a.device, (cols,)
    xt, rt, wt = _dtype(what, a), _dtype(what, r), _dtype(what, w_pre)
    gt, gp = binding.F8_BF16, None
    if gate is not None:
        gate_rows = rows if gate_rows is None else int(gate_rows)
        if gate_rows < 1 and rows > 0:
            raise ValueError(f"{what}: gate_rows must be at least 1")
        groups = -(-rows // max(gate_rows, 1))
        gt = _dtype(what, gate)
        if gate.dim() == 1 and groups <= 1:  # one gate for all rows
            gp = _ptr(what, "gate", gate, gate.dtype, shape, dev)
        else:
            gp = _ptr(what, "gate", gate, gate.dtype, (groups, cols), dev)
    return binding._ResidualNorm(
        int(kind), xt, rt, wt, gt, rows, cols, max(int(gate_rows or 1), 1), float(eps), float(scale),
        _ptr(what, "w_pre", w_pre, w_pre.dtype, shape, dev),
        _ptr(what, "b_pre", b_pre, w_pre.dtype, shape, dev),
        _ptr(what, "w_post", w_post, w_pre.dtype, shape, dev),
        _ptr(what, "b_post", b_post, w_pre.dtype, shape, dev), gp)


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
    all).  r may be fp32 beside a bf16 a.  stats fp32 [4, rows] is the backward's."""
    what = "f8_residual_norm_fwd"
    n = _residual_norm(what, a, r, w_pre, b_pre, w_post, b_post, gate, gate_rows, scale, kind, eps)
    shape, dev = a.shape, a.device
    r_out = _empty(shape, r.dtype, dev, stream) if r_out is None else r_out
    y = _empty(shape, a.dtype, dev, stream) if y is None else y
    stats = _empty((4, shape[0]), torch.float32, dev, stream) if stats is None else stats
    _call(what, stream, ctypes.byref(n), binding._ptr(a), _ptr(what, "r", r, r.dtype, shape, dev),
          _ptr(what, "r_out", r_out, r.dtype, shape, dev), _ptr(what, "y", y, a.dtype, shape, dev),
          _ptr(what, "stats", stats, torch.float32, (4, shape[0]), dev), _scalar(what, amax_out, dev))
    return r_out, y, stats


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
    shape, dev = a.shape, a.device
    cols = (shape[1],)
    like = {"da": (da, shape, a.dtype), "dr": (dr, shape, r_out.dtype),
            "dw_pre": (dw_pre, cols, w_pre.dtype), "db_pre": (db_pre, cols, w_pre.dtype),
            "dw_post": (dw_post, cols, w_pre.dtype), "db_post": (db_post, cols, w_pre.dtype),
            "dgate": (dgate, gate.shape if gate is not None else cols,
                      gate.dtype if gate is not None else w_pre.dtype)}
    if want is None:
        want = {"da", "dr", "dw_pre"}
        if kind == F8_LAYER_NORM:
            want.add("db_pre")
        if w_post is not None:
            want |= {"dw_post", "db_post"} if kind == F8_LAYER_NORM else {"dw_post"}
        if gate is not None:
            want.add("dgate")
    out, ptrs = [], []
    for name, (t, size, dtype) in like.items():
        if t is None and name in want:
            t = _empty(size, dtype, dev, stream)
        out.append(t)
        ptrs.append(_ptr(what, name, t, dtype, size, dev))
    grads = binding._ResidualNormGrads(*ptrs)
    if ws is None:
        ws = _empty(max(f8_residual_norm_bwd_workspace_bytes(*shape), 1), torch.uint8, dev, stream)
    _call(what, stream, ctypes.byref(n), _ptr(what, "dy", dy, a.dtype, shape, dev),
          _ptr(what, "dr_out", dr_out, r_out.dtype, shape, dev), binding._ptr(a),
          _ptr(what, "r_out", r_out, r_out.dtype, shape, dev),
          _ptr(what, "stats", stats, torch.float32, (4, shape[0]), dev), ctypes.byref(grads),
          *_bytes(what, ws, dev))
    return tuple(out)
