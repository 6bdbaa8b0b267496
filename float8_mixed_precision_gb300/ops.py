"""The operators around a Float8 linear, on torch tensors: the norm that
produces its input, the log probabilities read off a head linear's logits, and
the distillation loss against a teacher's top logits.

As in ``binding``, every function has the name of the C entry point of
include/f8.h that it calls and only checks and marshals its arguments: types,
shapes, devices and strides here, everything else in the C call.  Outputs and
workspaces that are not passed are allocated with torch, for the stream that
the call runs on.  There is no fallback.
"""
from __future__ import annotations

import torch

from . import binding
from .binding import F8_LAYER_NORM, _empty


# ---------------------------------------------------------------- norm
_DTYPES = {torch.bfloat16: binding.F8_BF16, torch.float32: binding.F8_F32}


def _dtype(what: str, t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"{what} takes bfloat16 or float32 tensors")
    return _DTYPES[t.dtype]


def _call(name: str, stream, *args) -> None:
    """The C call `name` on `stream`."""
    binding._check(getattr(binding.lib(), name)(*args, binding._stream(stream)), name)


def _ptr(what: str, name: str, t: torch.Tensor | None, dtype, shape: tuple, dev):
    """The pointer of `t` (None if not given): TypeError / ValueError unless it
    has this type, shape and device and is contiguous, as the C calls read or
    write it.  `dev` is the device of a tensor that binding._ptr or _rows
    takes, so it is the GPU's."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{what}: {name} must be {str(dtype).replace('torch.', '')}")
    if t.shape != shape:
        raise ValueError(f"{what}: {name} must have shape {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{what}: tensors on different devices")
    if not t.is_contiguous():
        raise ValueError("libf8 takes contiguous (row-major) tensors only")
    return t.data_ptr()


def _bytes(what: str, ws: torch.Tensor | None, dev):
    """The pointer and the size of a workspace, a tensor of bytes."""
    if ws is None:
        return None, 0
    return _ptr(what, "ws", ws, torch.uint8, (ws.numel(),), dev), ws.numel()


def _scalar(what: str, t: torch.Tensor | None, dev):
    """The pointer of one fp32 value (None if not given)."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() != 1:
        raise TypeError(f"{what}: amax_out must be one float32 value")
    if t.device != dev:
        raise ValueError(f"{what}: tensors on different devices")
    return t.data_ptr()


def _norm_params(what: str, x, w, b):
    """Types and pointers of x, w and b."""
    if x.dim() != 2:
        raise TypeError(f"{what} takes a 2-D input")
    cols, dev = (x.shape[1],), x.device
    wt = _dtype(what, w)
    wp, bp = _ptr(what, "w", w, w.dtype, cols, dev), _ptr(what, "b", b, w.dtype, cols, dev)
    return _dtype(what, x), wt, binding._ptr(x), wp, bp


def f8_norm_fwd(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None = None,
                kind: int = F8_LAYER_NORM, eps: float = 1e-5, y: torch.Tensor | None = None,
                mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                amax_out: torch.Tensor | None = None, stream=None):
    """Layer norm or RMS norm of the rows of a 2-D bf16 or fp32 tensor;
    returns (y, mean, rstd), mean None for F8_RMS_NORM.  `amax_out` (fp32
    scalar, bf16 inputs) receives max |y|, ready for f8_cast_transpose."""
    what = "f8_norm_fwd"
    xt, wt, xp, wp, bp = _norm_params(what, x, w, b)
    rows, cols = shape = x.shape
    dev = x.device
    y = _empty(shape, x.dtype, dev, stream) if y is None else y
    if mean is None and kind == F8_LAYER_NORM:
        mean = _empty(rows, torch.float32, dev, stream)
    rstd = _empty(rows, torch.float32, dev, stream) if rstd is None else rstd
    _call(what, stream, xp, xt, wp, bp, wt, int(kind), rows, cols, float(eps),
          _ptr(what, "y", y, x.dtype, shape, dev),
          _ptr(what, "mean", mean, torch.float32, (rows,), dev),
          _ptr(what, "rstd", rstd, torch.float32, (rows,), dev), _scalar(what, amax_out, dev))
    return y, (mean if kind == F8_LAYER_NORM else None), rstd


def f8_norm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return int(binding.lib().f8_norm_bwd_workspace_bytes(rows, cols))


def f8_norm_bwd(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, mean: torch.Tensor | None,
                rstd: torch.Tensor, kind: int = F8_LAYER_NORM, dx: torch.Tensor | None = None,
                dw: torch.Tensor | None = None, db: torch.Tensor | None = None,
                ws: torch.Tensor | None = None, want_dx: bool = True, want_dw: bool = True,
                want_db: bool | None = None, stream=None):
    """(dx, dw, db) of f8_norm_fwd for the gradient dy of y; db is formed by
    default for F8_LAYER_NORM (`want_db`)."""
    what = "f8_norm_bwd"
    xt, wt, xp, wp, _ = _norm_params(what, x, w, None)
    rows, cols = shape = x.shape
    dev = x.device
    if want_db is None:
        want_db = kind == F8_LAYER_NORM
    dx = _empty(shape, x.dtype, dev, stream) if dx is None and want_dx else dx
    dw = _empty(cols, w.dtype, dev, stream) if dw is None and want_dw else dw
    db = _empty(cols, w.dtype, dev, stream) if db is None and want_db else db
    args = (_ptr(what, "dy", dy, x.dtype, shape, dev), xp, xt, wp, wt,
            _ptr(what, "mean", mean, torch.float32, (rows,), dev),
            _ptr(what, "rstd", rstd, torch.float32, (rows,), dev), int(kind), rows, cols,
            _ptr(what, "dx", dx, x.dtype, shape, dev), _ptr(what, "dw", dw, w.dtype, (cols,), dev),
            _ptr(what, "db", db, w.dtype, (cols,), dev))
    if ws is None and (dw is not None or db is not None):
        ws = _empty(max(f8_norm_bwd_workspace_bytes(rows, cols), 1), torch.uint8, dev, stream)
    _call(what, stream, *args, *_bytes(what, ws, dev))
    return dx, dw, db


def f8_quantize_norm(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None = None,
                     kind: int = F8_LAYER_NORM, eps: float = 1e-5, y: torch.Tensor | None = None,
                     mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                     amax_out=None, scale_out=None, q=None, q_t=None, ws=None, stream=None):
    """The norm of a 2-D bf16 tensor with its amax from the producing pass,
    then its E4M3 cast: returns (q, q_t, scale, amax, y, mean, rstd)."""
    what = "f8_quantize_norm"
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{what} takes a bf16 input")
    _, wt, xp, wp, bp = _norm_params(what, x, w, b)
    rows, cols = shape = x.shape
    dev = x.device
    y = _empty(shape, x.dtype, dev, stream) if y is None else y
    if mean is None and kind == F8_LAYER_NORM:
        mean = _empty(rows, torch.float32, dev, stream)
    rstd = _empty(rows, torch.float32, dev, stream) if rstd is None else rstd
    amax_out = _empty((), torch.float32, dev, stream) if amax_out is None else amax_out
    scale_out = _empty((), torch.float32, dev, stream) if scale_out is None else scale_out
    q = _empty((rows, cols), torch.uint8, dev, stream) if q is None else q
    q_t = _empty((cols, rows), torch.uint8, dev, stream) if q_t is None else q_t
    if ws is None:
        ws = _empty(binding.f8_quantize_workspace_bytes(), torch.uint8, dev, stream)
    _call(what, stream, xp, wp, bp, wt, int(kind), rows, cols, float(eps),
          _ptr(what, "y", y, x.dtype, shape, dev),
          _ptr(what, "mean", mean, torch.float32, (rows,), dev),
          _ptr(what, "rstd", rstd, torch.float32, (rows,), dev), _scalar(what, amax_out, dev),
          _scalar(what, scale_out, dev), _ptr(what, "q", q, torch.uint8, (rows, cols), dev),
          _ptr(what, "q_t", q_t, torch.uint8, (cols, rows), dev), *_bytes(what, ws, dev))
    return q, q_t, scale_out, amax_out, y, (mean if kind == F8_LAYER_NORM else None), rstd


# ---------------------------------------------------------------- logits
def _on_device(t: torch.Tensor) -> bool:
    return t.is_cuda


def _rows(what: str, name: str, t: torch.Tensor):
    """(pointer, row stride) of a 2-D tensor whose rows are dense but may lie
    apart (a view of the first columns of a wider buffer)."""
    if t.dim() != 2:
        raise TypeError(f"{what}: {name} must be 2-D")
    if not _on_device(t):
        raise ValueError("libf8 takes device tensors only")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the columns of {name} must be contiguous")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{what}: the rows of {name} overlap")
    return t.data_ptr(), ld


def _dlogits(what: str, logits: torch.Tensor, dlogits: torch.Tensor | None, stream):
    """The gradient buffer (one row per row of logits, its columns past the
    vocabulary set to zero by the call) and its pointer and row stride."""
    rows, vocab = logits.shape
    if dlogits is None:
        dlogits = _empty((rows, vocab), logits.dtype, logits.device, stream)
    if dlogits.device != logits.device:
        raise ValueError(f"{what}: tensors on different devices")
    if dlogits.dtype != logits.dtype:
        raise TypeError(f"{what}: dlogits must have the type of logits")
    if dlogits.dim() != 2 or dlogits.shape[0] != rows or dlogits.shape[1] < vocab:
        raise ValueError(f"{what}: dlogits must be [rows, vocab] or wider")
    return dlogits, binding._ptr(dlogits), dlogits.shape[1]


def f8_token_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top_k: int = 0,
                      temperature: float = 1.0, logp: torch.Tensor | None = None,
                      entropy: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      top_ids: torch.Tensor | None = None, top_logp: torch.Tensor | None = None,
                      stream=None):
    """Per row of logits [rows, vocab] (bf16 or fp32, rows may lie apart):
    (logp of `tokens`, entropy, log-sum-exp, top_ids, top_logp), all under
    logits / temperature; logp is None without tokens, the last two without
    top_k.  A negative token marks a row that is ignored."""
    what = "f8_token_logprobs"
    p, ld = _rows(what, "logits", logits)
    rows, vocab = logits.shape
    dev = logits.device
    f32 = (torch.float32, dev, stream)
    if tokens is not None and logp is None:
        logp = _empty(rows, *f32)
    entropy = _empty(rows, *f32) if entropy is None else entropy
    lse = _empty(rows, *f32) if lse is None else lse
    if top_k and top_ids is None:
        top_ids = _empty((rows, top_k), torch.int32, dev, stream)
    if top_k and top_logp is None:
        top_logp = _empty((rows, top_k), *f32)
    _call(what, stream, p, _dtype(what, logits), rows, vocab, ld,
          _ptr(what, "tokens", tokens, torch.int64, (rows,), dev), float(temperature), int(top_k),
          _ptr(what, "logp", logp, torch.float32, (rows,), dev),
          _ptr(what, "entropy", entropy, torch.float32, (rows,), dev),
          _ptr(what, "lse", lse, torch.float32, (rows,), dev),
          _ptr(what, "top_ids", top_ids, torch.int32, (rows, top_k), dev),
          _ptr(what, "top_logp", top_logp, torch.float32, (rows, top_k), dev))
    return logp, entropy, lse, top_ids, top_logp


def f8_token_logprobs_bwd(logits: torch.Tensor, tokens: torch.Tensor | None, lse: torch.Tensor,
                          entropy: torch.Tensor | None, dlogp: torch.Tensor | None,
                          dentropy: torch.Tensor | None, temperature: float = 1.0,
                          dlogits: torch.Tensor | None = None,
                          amax_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of logp and entropy to the logits, in `dlogits` (which may
    be wider than the vocabulary: its further columns are set to zero)."""
    what = "f8_token_logprobs_bwd"
    p, ld = _rows(what, "logits", logits)
    rows, vocab = logits.shape
    dev = logits.device
    dlogits, dp, ldd = _dlogits(what, logits, dlogits, stream)
    _call(what, stream, p, _dtype(what, logits), rows, vocab, ld,
          _ptr(what, "tokens", tokens, torch.int64, (rows,), dev),
          _ptr(what, "lse", lse, torch.float32, (rows,), dev),
          _ptr(what, "entropy", entropy, torch.float32, (rows,), dev),
          _ptr(what, "dlogp", dlogp, torch.float32, (rows,), dev),
          _ptr(what, "dentropy", dentropy, torch.float32, (rows,), dev), float(temperature), dp,
          ldd, _scalar(what, amax_out, dev))
    return dlogits


def _slots(what: str, logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor):
    """The pointers of the slots' ids and values, and their number."""
    if ids.dim() != 2:
        raise TypeError(f"{what}: ids must be 2-D")
    shape, dev = (logits.shape[0], ids.shape[1]), logits.device
    return (_ptr(what, "ids", ids, torch.int32, shape, dev),
            _ptr(what, "values", values, torch.float32, shape, dev), shape[1])


def f8_distill_fwd(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor,
                   temperature: float = 1.0, tail: bool = False, loss: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, rest: torch.Tensor | None = None, stream=None):
    """The distillation loss of each row of logits [rows, vocab] against the
    teacher's slots ids, values [rows, k]: (loss, lse, rest), the last two for
    f8_distill_bwd (rest None without `tail`)."""
    what = "f8_distill_fwd"
    p, ld = _rows(what, "logits", logits)
    rows, vocab = logits.shape
    dev = logits.device
    slots = _slots(what, logits, ids, values)
    f32 = (torch.float32, dev, stream)
    loss = _empty(rows, *f32) if loss is None else loss
    lse = _empty(rows, *f32) if lse is None else lse
    if tail and rest is None:
        rest = _empty(rows, *f32)
    _call(what, stream, p, _dtype(what, logits), rows, vocab, ld, *slots, float(temperature),
          int(bool(tail)), _ptr(what, "loss", loss, torch.float32, (rows,), dev),
          _ptr(what, "lse", lse, torch.float32, (rows,), dev),
          _ptr(what, "rest", rest, torch.float32, (rows,), dev))
    return loss, lse, (rest if tail else None)


def f8_distill_bwd(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor, lse: torch.Tensor,
                   rest: torch.Tensor | None, dloss: torch.Tensor, temperature: float = 1.0,
                   tail: bool = False, dlogits: torch.Tensor | None = None,
                   amax_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dlogits of f8_distill_fwd for the gradient dloss [rows] of the loss."""
    what = "f8_distill_bwd"
    p, ld = _rows(what, "logits", logits)
    rows, vocab = logits.shape
    dev = logits.device
    slots = _slots(what, logits, ids, values)
    dlogits, dp, ldd = _dlogits(what, logits, dlogits, stream)
    _call(what, stream, p, _dtype(what, logits), rows, vocab, ld, *slots, float(temperature),
          int(bool(tail)), _ptr(what, "lse", lse, torch.float32, (rows,), dev),
          _ptr(what, "rest", rest, torch.float32, (rows,), dev),
          _ptr(what, "dloss", dloss, torch.float32, (rows,), dev), dp, ldd,
          _scalar(what, amax_out, dev))
    return dlogits


def f8_distill_fwd_bwd(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor,
                       dloss: torch.Tensor, temperature: float = 1.0, tail: bool = False,
                       loss: torch.Tensor | None = None, dlogits: torch.Tensor | None = None,
                       amax_out: torch.Tensor | None = None, stream=None):
    """(loss, dlogits) in one pass over the logits, for callers that know the
    gradient dloss [rows] of the loss beforehand."""
    what = "f8_distill_fwd_bwd"
    p, ld = _rows(what, "logits", logits)
    rows, vocab = logits.shape
    dev = logits.device
    slots = _slots(what, logits, ids, values)
    dlogits, dp, ldd = _dlogits(what, logits, dlogits, stream)
    loss = _empty(rows, torch.float32, dev, stream) if loss is None else loss
    _call(what, stream, p, _dtype(what, logits), rows, vocab, ld, *slots, float(temperature),
          int(bool(tail)), _ptr(what, "dloss", dloss, torch.float32, (rows,), dev),
          _ptr(what, "loss", loss, torch.float32, (rows,), dev), dp, ldd,
          _scalar(what, amax_out, dev))
    return loss, dlogits
