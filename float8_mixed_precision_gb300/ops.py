"""The operators around a Float8 linear, on torch tensors: the norm that
produces its input, the log probabilities read off a head linear's logits, and
the distillation loss against a teacher's top logits.

As in ``binding``, every function has the name of the C entry point of
include/f8.h that it calls and only checks and marshals its arguments: types,
shapes, devices and strides here, everything else in the C call.  Outputs and
workspaces that are not passed are allocated with torch.  There is no fallback.
"""
from __future__ import annotations

import torch

from . import binding
from .binding import F8_LAYER_NORM


# ---------------------------------------------------------------- norm
_DTYPES = {torch.bfloat16: binding.F8_BF16, torch.float32: binding.F8_F32}


def _dtype(what: str, t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"{what} takes bfloat16 or float32 tensors")
    return _DTYPES[t.dtype]


def _call(name: str, stream, *args) -> None:
    """The C call `name` with tensors as device pointers, on `stream`."""
    ptr = binding._ptr
    args = [ptr(a) if isinstance(a, torch.Tensor) else a for a in args]
    binding._check(getattr(binding.lib(), name)(*args, binding._stream(stream)), name)


def _like(what: str, name: str, t: torch.Tensor | None, dtype, shape: tuple, dev) -> None:
    """TypeError / ValueError unless `t` (when given) has this type, shape and
    device: the C calls write or read it as such."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{what}: {name} must be {str(dtype).replace('torch.', '')}")
    if t.shape != shape:
        raise ValueError(f"{what}: {name} must have shape {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{what}: tensors on different devices")


def _same_device(what: str, dev, t: torch.Tensor | None) -> None:
    if t is not None and t.device != dev:
        raise ValueError(f"{what}: tensors on different devices")


def _amax(what: str, t: torch.Tensor | None, dev) -> None:
    if t is None:
        return
    if t.dtype != torch.float32 or t.numel() != 1:
        raise TypeError(f"{what}: amax_out must be one float32 value")
    if t.device != dev:
        raise ValueError(f"{what}: tensors on different devices")


def _norm_params(what: str, x, w, b):
    if x.dim() != 2:
        raise TypeError(f"{what} takes a 2-D input")
    cols, dev = (x.shape[1],), x.device
    _like(what, "w", w, w.dtype, cols, dev)
    _like(what, "b", b, w.dtype, cols, dev)
    return _dtype(what, x), _dtype(what, w)


def f8_norm_fwd(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None = None,
                kind: int = F8_LAYER_NORM, eps: float = 1e-5, y: torch.Tensor | None = None,
                mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                amax_out: torch.Tensor | None = None, stream=None):
    """Layer norm or RMS norm of the rows of a 2-D bf16 or fp32 tensor;
    returns (y, mean, rstd), mean None for F8_RMS_NORM.  `amax_out` (fp32
    scalar, bf16 inputs) receives max |y|, ready for f8_cast_transpose."""
    xt, wt = _norm_params("f8_norm_fwd", x, w, b)
    rows, cols = x.shape
    dev = x.device
    y = torch.empty_like(x) if y is None else y
    if mean is None and kind == F8_LAYER_NORM:
        mean = torch.empty(rows, dtype=torch.float32, device=dev)
    rstd = torch.empty(rows, dtype=torch.float32, device=dev) if rstd is None else rstd
    _like("f8_norm_fwd", "y", y, x.dtype, x.shape, dev)
    _like("f8_norm_fwd", "mean", mean, torch.float32, (rows,), dev)
    _like("f8_norm_fwd", "rstd", rstd, torch.float32, (rows,), dev)
    _amax("f8_norm_fwd", amax_out, dev)
    _call("f8_norm_fwd", stream, x, xt, w, b, wt, int(kind), rows, cols, float(eps), y, mean,
          rstd, amax_out)
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
    xt, wt = _norm_params("f8_norm_bwd", x, w, None)
    rows, cols = x.shape
    dev = x.device
    _like("f8_norm_bwd", "dy", dy, x.dtype, x.shape, dev)
    _like("f8_norm_bwd", "mean", mean, torch.float32, (rows,), dev)
    _like("f8_norm_bwd", "rstd", rstd, torch.float32, (rows,), dev)
    if want_db is None:
        want_db = kind == F8_LAYER_NORM
    dx = torch.empty_like(x) if dx is None and want_dx else dx
    dw = torch.empty_like(w) if dw is None and want_dw else dw
    db = torch.empty_like(w) if db is None and want_db else db
    _like("f8_norm_bwd", "dx", dx, x.dtype, x.shape, dev)
    _like("f8_norm_bwd", "dw", dw, w.dtype, (cols,), dev)
    _like("f8_norm_bwd", "db", db, w.dtype, (cols,), dev)
    if ws is None and (dw is not None or db is not None):
        ws = torch.empty(max(f8_norm_bwd_workspace_bytes(rows, cols), 1), dtype=torch.uint8, device=dev)
    _same_device("f8_norm_bwd", dev, ws)
    _call("f8_norm_bwd", stream, dy, x, xt, w, wt, mean, rstd, int(kind), rows, cols, dx, dw,
          db, ws, ws.numel() if ws is not None else 0)
    return dx, dw, db


def f8_quantize_norm(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None = None,
                     kind: int = F8_LAYER_NORM, eps: float = 1e-5, y: torch.Tensor | None = None,
                     mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                     amax_out=None, scale_out=None, q=None, q_t=None, ws=None, stream=None):
    """The norm of a 2-D bf16 tensor with its amax from the producing pass,
    then its E4M3 cast: returns (q, q_t, scale, amax, y, mean, rstd)."""
    if x.dtype != torch.bfloat16:
        raise TypeError("f8_quantize_norm takes a bf16 input")
    _, wt = _norm_params("f8_quantize_norm", x, w, b)
    rows, cols = x.shape
    dev = x.device
    y = torch.empty_like(x) if y is None else y
    if mean is None and kind == F8_LAYER_NORM:
        mean = torch.empty(rows, dtype=torch.float32, device=dev)
    rstd = torch.empty(rows, dtype=torch.float32, device=dev) if rstd is None else rstd
    amax_out = torch.empty((), dtype=torch.float32, device=dev) if amax_out is None else amax_out
    scale_out = torch.empty((), dtype=torch.float32, device=dev) if scale_out is None else scale_out
    q = torch.empty((rows, cols), dtype=torch.uint8, device=dev) if q is None else q
    q_t = torch.empty((cols, rows), dtype=torch.uint8, device=dev) if q_t is None else q_t
    if ws is None:
        ws = torch.empty(binding.f8_quantize_workspace_bytes(), dtype=torch.uint8, device=dev)
    _like("f8_quantize_norm", "y", y, x.dtype, x.shape, dev)
    _like("f8_quantize_norm", "mean", mean, torch.float32, (rows,), dev)
    _like("f8_quantize_norm", "rstd", rstd, torch.float32, (rows,), dev)
    _like("f8_quantize_norm", "q", q, torch.uint8, (rows, cols), dev)
    _like("f8_quantize_norm", "q_t", q_t, torch.uint8, (cols, rows), dev)
    _amax("f8_quantize_norm", amax_out, dev)
    _amax("f8_quantize_norm", scale_out, dev)
    _same_device("f8_quantize_norm", dev, ws)
    _call("f8_quantize_norm", stream, x, w, b, wt, int(kind), rows, cols, float(eps), y, mean,
          rstd, amax_out, scale_out, q, q_t, ws, ws.numel())
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


def _dlogits(what: str, logits: torch.Tensor, dlogits: torch.Tensor | None):
    """The gradient buffer (one row per row of logits, its columns past the
    vocabulary set to zero by the call) and its pointer and row stride."""
    rows, vocab = logits.shape
    if dlogits is None:
        dlogits = torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
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
    f32 = dict(dtype=torch.float32, device=dev)
    if tokens is not None and logp is None:
        logp = torch.empty(rows, **f32)
    entropy = torch.empty(rows, **f32) if entropy is None else entropy
    lse = torch.empty(rows, **f32) if lse is None else lse
    if top_k and top_ids is None:
        top_ids = torch.empty((rows, top_k), dtype=torch.int32, device=logits.device)
    if top_k and top_logp is None:
        top_logp = torch.empty((rows, top_k), **f32)
    _like(what, "tokens", tokens, torch.int64, (rows,), dev)
    for n, t in (("logp", logp), ("entropy", entropy), ("lse", lse)):
        _like(what, n, t, torch.float32, (rows,), dev)
    _like(what, "top_ids", top_ids, torch.int32, (rows, top_k), dev)
    _like(what, "top_logp", top_logp, torch.float32, (rows, top_k), dev)
    _call("f8_token_logprobs", stream, p, _dtype(what, logits), rows, vocab, ld, tokens,
          float(temperature), int(top_k), logp, entropy, lse, top_ids, top_logp)
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
    dlogits, dp, ldd = _dlogits(what, logits, dlogits)
    _like(what, "tokens", tokens, torch.int64, (rows,), dev)
    for n, t in (("lse", lse), ("entropy", entropy), ("dlogp", dlogp), ("dentropy", dentropy)):
        _like(what, n, t, torch.float32, (rows,), dev)
    _amax(what, amax_out, dev)
    _call("f8_token_logprobs_bwd", stream, p, _dtype(what, logits), rows, vocab, ld, tokens,
          lse, entropy, dlogp, dentropy, float(temperature), dp, ldd, amax_out)
    return dlogits


def _slots(what: str, logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor) -> int:
    if ids.dim() != 2:
        raise TypeError(f"{what}: ids must be 2-D")
    k, dev = ids.shape[1], logits.device
    _like(what, "ids", ids, torch.int32, (logits.shape[0], k), dev)
    _like(what, "values", values, torch.float32, (logits.shape[0], k), dev)
    return k


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
    k = _slots(what, logits, ids, values)
    f32 = dict(dtype=torch.float32, device=logits.device)
    loss = torch.empty(rows, **f32) if loss is None else loss
    lse = torch.empty(rows, **f32) if lse is None else lse
    if tail and rest is None:
        rest = torch.empty(rows, **f32)
    for n, t in (("loss", loss), ("lse", lse), ("rest", rest)):
        _like(what, n, t, torch.float32, (rows,), dev)
    _call("f8_distill_fwd", stream, p, _dtype(what, logits), rows, vocab, ld, ids, values, k,
          float(temperature), int(bool(tail)), loss, lse, rest)
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
    k = _slots(what, logits, ids, values)
    dlogits, dp, ldd = _dlogits(what, logits, dlogits)
    for n, t in (("lse", lse), ("rest", rest), ("dloss", dloss)):
        _like(what, n, t, torch.float32, (rows,), dev)
    _amax(what, amax_out, dev)
    _call("f8_distill_bwd", stream, p, _dtype(what, logits), rows, vocab, ld, ids, values, k,
          float(temperature), int(bool(tail)), lse, rest, dloss, dp, ldd, amax_out)
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
    k = _slots(what, logits, ids, values)
    dlogits, dp, ldd = _dlogits(what, logits, dlogits)
    loss = torch.empty(rows, dtype=torch.float32, device=logits.device) if loss is None else loss
    for n, t in (("loss", loss), ("dloss", dloss)):
        _like(what, n, t, torch.float32, (rows,), dev)
    _amax(what, amax_out, dev)
    _call("f8_distill_fwd_bwd", stream, p, _dtype(what, logits), rows, vocab, ld, ids, values,
          k, float(temperature), int(bool(tail)), dloss, loss, dp, ldd, amax_out)
    return loss, dlogits
