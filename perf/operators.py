"""Operators around a Float8 training linear: normalisation, token log probabilities and top-logit distillation.

What is measured, case by case: the norm in front of a block's linears or of the head (layer norm or RMS norm, forward and
backward with the reduction of the weight's gradient), the log probabilities of given tokens with their entropy and the
top alternatives (forward, and the gradient for policy losses), and the distillation loss against a teacher's top
logits (forward, backward, and both in one pass for training loops that know the rows' weights).

``run`` computes the plain form (elementary torch operations in 32 bits, rounded once) unless ``own`` is set, and then makes
the framework's calls on the same state.
"""
import math

import torch

own = False

NEG_INF = float("-inf")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NORM_EPS = 1e-5


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the final norm of eight sequences that decode one token each: one launch's latency
        dict(name="norm_fwd_decode", op="norm_fwd", kind="rms", dtype="bf16", rows=8, cols=4096),
        # the norm in front of the q, k and v projections of the 8B block, at the block's 8192 tokens
        dict(name="norm_fwd_block", op="norm_fwd", kind="layer", dtype="bf16", rows=8192, cols=4096),
        # its backward pass, with the weight's and the bias's gradients
        dict(name="norm_bwd_block", op="norm_bwd", kind="layer", dtype="bf16", rows=8192, cols=4096),
        # a ragged batch, and a width that no vector divides
        dict(name="norm_bwd_odd", op="norm_bwd", kind="rms", dtype="bf16", rows=1999, cols=5003),
        # one decoding step that reports its tokens' log probabilities and twenty alternatives
        dict(name="logprobs_decode", op="logprobs", dtype="bf16", rows=4, vocab=131072, pad=0, k=20,
             temperature=1.0, masked=0.0, ignored=0),
        # scoring a batch of sequences
        dict(name="logprobs_score", op="logprobs", dtype="bf16", rows=4096, vocab=131072, pad=0, k=8,
             temperature=1.0, masked=0.0, ignored=100),
        # 32-bit logits of an odd vocabulary with forbidden tokens, at a sampling temperature: a teacher's pass
        dict(name="logprobs_teacher_odd", op="logprobs", dtype="f32", rows=333, vocab=50003, pad=0, k=64,
             temperature=0.7, masked=0.1, ignored=13),
        # a policy loss with an entropy bonus, back to the logits
        dict(name="logprobs_bwd_policy", op="logprobs_bwd", dtype="bf16", rows=2048, vocab=65536, pad=0, k=0,
             temperature=0.8, masked=0.0, ignored=50),
        # a training step of the student: loss and gradient together
        dict(name="distill_train", op="distill_train", dtype="bf16", rows=4096, vocab=131072, pad=0, k=64,
             temperature=2.0, tail=False, ignored=100),
        # the same on a padded odd vocabulary, with the mass outside the teacher's list as one more class
        dict(name="distill_train_tail_odd", op="distill_train", dtype="bf16", rows=777, vocab=50003, pad=13, k=32,
             temperature=1.0, tail=True, ignored=20),
        # the loss alone, as in an evaluation
        dict(name="distill_eval", op="distill_fwd", dtype="f32", rows=512, vocab=32768, pad=0, k=128,
             temperature=1.0, tail=True, ignored=0),
        # the backward pass alone, as autograd calls it
        dict(name="distill_bwd", op="distill_bwd", dtype="bf16", rows=1024, vocab=131072, pad=0, k=16,
             temperature=1.0, tail=False, ignored=10),
    ]


OPS = ("norm_fwd", "norm_bwd", "logprobs", "logprobs_bwd", "distill_train", "distill_fwd", "distill_bwd")
MOST_BYTES = 4096 * 131072 * 4


def _spread(rng, lo, hi):
    """A whole number, its logarithm spread over [lo, hi]; a third are multiples of 128, the others as they fall."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 1 / 3 and n >= 128:
        n -= n % 128
    if n == 3072:
        n += 1
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    size = 2 if dtype == "bf16" else 4
    if op.startswith("norm"):
        cols = _spread(rng, 64, 16384)
        if rng.random() < 0.5 and cols % 8 and (cols + 8 - cols % 8) != 3072:
            cols += 8 - cols % 8
        return dict(op=op, kind=rng.choice(("layer", "rms")), dtype=dtype,
                    rows=_spread(rng, 1, min(16384, MOST_BYTES // (4 * cols * size))), cols=cols)
    vocab = _spread(rng, 1000, 200000)
    rows = _spread(rng, 1, max(2, min(8192, MOST_BYTES // (4 * vocab * size))))
    case = dict(op=op, dtype=dtype, rows=rows, vocab=vocab, pad=rng.choice((0, 0, -vocab % 16)), k=0,
                temperature=rng.choice((1.0, 1.0, 0.7, 2.0)), ignored=rng.choice((0, rows // 20, rows // 4)))
    if op == "logprobs":
        case["k"] = rng.choice((0, 1, 5, 20, 64, 100))
    if op.startswith("logprobs"):
        case["masked"] = rng.choice((0.0, 0.0, 0.1, 0.5))
    else:
        case["k"] = _spread(rng, 1, 128)
        case["tail"] = rng.random() < 0.5
    return case


def work(case):
    """Each input read once and each output written once; a row that is ignored is not read."""
    size = 2 if case["dtype"] == "bf16" else 4
    rows, op = case["rows"], case["op"]
    if op.startswith("norm"):
        cols = case["cols"]
        params = 2 if case["kind"] == "layer" else 1
        stats = 4 * params * rows
        if op == "norm_fwd":
            return {"bytes": 2 * rows * cols * size + params * cols * size + stats, "flops": 8 * rows * cols}
        return {"bytes": 3 * rows * cols * size + (1 + params) * cols * size + stats, "flops": 12 * rows * cols}
    vocab, k = case["vocab"], case["k"]
    read = (rows - case["ignored"]) * vocab * size
    wrote = rows * (vocab + case["pad"]) * size
    if op == "logprobs":
        return {"bytes": read + rows * (8 + 12 + 8 * k), "flops": 6 * rows * vocab}
    if op == "logprobs_bwd":
        return {"bytes": read + wrote + rows * (8 + 16), "flops": 8 * rows * vocab}
    small = rows * (8 * k + (12 if case["tail"] else 8))
    if op == "distill_fwd":
        return {"bytes": read + small, "flops": 5 * rows * vocab}
    if op == "distill_bwd":
        return {"bytes": read + wrote + small, "flops": 5 * rows * vocab}
    return {"bytes": read + wrote + small, "flops": 9 * rows * vocab}


# ---------------------------------------------------------------- inputs
def _logits(case, gen):
    """[rows, vocab + pad] logits as a head gives them: a common bias per token over which each row spreads, and in some
    rows a few tokens far above the rest.  Forbidden tokens are -inf in every row; the padding is not part of any row."""
    rows, vocab, pad = case["rows"], case["vocab"], case["pad"]
    dt = TYPES[case["dtype"]]
    full = torch.empty((rows, vocab + pad), dtype=dt, device="cuda")
    bias = 1.5 * torch.randn((vocab,), generator=gen, device="cuda")
    if case.get("masked"):
        gone = torch.rand((vocab,), generator=gen, device="cuda") < case["masked"]
        gone[: min(vocab, 512)] = False
        bias = torch.where(gone, torch.full_like(bias, NEG_INF), bias)
    z = torch.randn((rows, vocab), generator=gen, device="cuda")
    full[:, :vocab] = z.mul_(2.0).add_(bias)
    full[:, vocab:] = 0
    peak = torch.randint(0, min(vocab, 512), (rows, 4), generator=gen, device="cuda")
    up = full.gather(1, peak).float() + torch.rand((rows, 4), generator=gen, device="cuda") * 9.0
    full.scatter_(1, peak, up.to(dt))
    return full


def _ignored(case, gen):
    """Which rows are padding of the batch."""
    out = torch.zeros((case["rows"],), dtype=torch.bool, device="cuda")
    out[torch.randperm(case["rows"], generator=gen, device="cuda")[: case["ignored"]]] = True
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    op, rows, dt = case["op"], case["rows"], TYPES[case["dtype"]]
    s = {"case": case}
    if op.startswith("norm"):
        cols = case["cols"]
        x = torch.randn((rows, cols), generator=gen, device="cuda")
        x = x * (0.5 + 2.0 * torch.rand((cols,), generator=gen, device="cuda")) + 0.3
        s["x"] = x.to(dt)
        s["w"] = (1.0 + 0.2 * torch.randn((cols,), generator=gen, device="cuda")).to(dt)
        layer = case["kind"] == "layer"
        s["b"] = (0.1 * torch.randn((cols,), generator=gen, device="cuda")).to(dt) if layer else None
        f32 = dict(dtype=torch.float32, device="cuda")
        if op == "norm_bwd":
            s["dy"] = (torch.randn((rows, cols), generator=gen, device="cuda") * 0.01).to(dt)
            xd = s["x"].float()
            mean = xd.mean(1) if layer else torch.zeros((rows,), **f32)
            s["rstd"] = ((xd - mean[:, None]).square().mean(1) + NORM_EPS).rsqrt()
            s["mean"] = mean if layer else None
            # a training program's gradient buffers
            s["out"] = {"dx": torch.empty_like(s["x"]), "dw": torch.empty_like(s["w"]),
                        "db": torch.empty_like(s["w"]) if layer else None}
        else:
            s["out"] = {"y": torch.empty_like(s["x"]), "mean": torch.empty((rows,), **f32) if layer else None,
                        "rstd": torch.empty((rows,), **f32)}
        return s
    vocab, k = case["vocab"], case["k"]
    s["full"] = _logits(case, gen)
    s["logits"] = s["full"][:, :vocab]
    skip = _ignored(case, gen)
    f32 = dict(dtype=torch.float32, device="cuda")
    tau = case["temperature"]
    if op.startswith("logprobs"):
        tokens = torch.randint(0, min(vocab, 512), (rows,), generator=gen, device="cuda")
        s["tokens"] = torch.where(skip, torch.full_like(tokens, -1), tokens)
        if op == "logprobs":
            i32 = dict(dtype=torch.int32, device="cuda")
            s["out"] = {"logp": torch.empty((rows,), **f32), "entropy": torch.empty((rows,), **f32),
                        "lse": torch.empty((rows,), **f32), "top_ids": torch.empty((rows, k), **i32) if k else None,
                        "top_logp": torch.empty((rows, k), **f32) if k else None}
            return s
        z = s["logits"].float() / tau  # what the forward pass kept
        lse = torch.logsumexp(z, 1)
        p = torch.exp(z - lse[:, None])
        ent = lse - torch.where(p > 0, p * z, torch.zeros_like(p)).sum(1)
        s["lse"] = torch.where(skip, torch.zeros((), **f32), lse)
        s["entropy"] = torch.where(skip, torch.zeros((), **f32), ent)
        s["dlogp"] = torch.randn((rows,), generator=gen, device="cuda") / rows
        s["dentropy"] = torch.full((rows,), -0.01 / rows, **f32)
        s["dlogits"] = torch.empty_like(s["full"])
        return s
    # the teacher's list: distinct ids, one in each of k stretches of the vocabulary, near the student's own logits
    wide = vocab // k
    ids = torch.arange(k, device="cuda") * wide + torch.randint(0, wide, (rows, k), generator=gen, device="cuda")
    t = s["logits"].gather(1, ids).float() / tau + torch.randn((rows, k), generator=gen, device="cuda")
    t = t + 6.0 * torch.rand((rows, k), generator=gen, device="cuda")
    if case["tail"]:  # log probabilities at this temperature that leave some mass outside the list
        mass = 0.6 + 0.39 * torch.rand((rows, 1), generator=gen, device="cuda")
        t = torch.log_softmax(t, 1) + mass.log()
    else:
        t = t * tau
    short = torch.rand((rows, k), generator=gen, device="cuda") < 0.02  # slots that a shorter list left empty
    short[:, 0] = False
    s["ids"] = torch.where(short | skip[:, None], torch.full_like(ids, -1), ids).to(torch.int32)
    s["values"] = t
    s["dloss"] = torch.where(skip, torch.zeros((), **f32), torch.full((rows,), 1.0 / rows, **f32))
    s["loss"] = torch.empty((rows,), **f32)
    s["lse"] = torch.empty((rows,), **f32)
    s["rest"] = torch.empty((rows,), **f32) if case["tail"] else None
    if op != "distill_fwd":
        s["dlogits"] = torch.empty_like(s["full"])
    if op == "distill_bwd":
        live = (s["ids"] >= 0).any(1)
        z = s["logits"].float() / tau
        lse = torch.logsumexp(z, 1)
        s["lse"] = torch.where(live, lse, torch.zeros((), **f32))
        if case["tail"]:
            p = torch.cat((torch.exp(z - lse[:, None]), torch.zeros((rows, 1), **f32)), 1)
            p.scatter_(1, torch.where(s["ids"] < 0, vocab, s["ids"]).long(), 0.0)
            s["rest"] = torch.where(live, p.sum(1), torch.zeros((), **f32))
    return s


# ---------------------------------------------------------------- the two forms
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import float8_mixed_precision_gb300 as f8
    c = s["case"]
    op = c["op"]
    if op.startswith("norm"):
        kind = f8.F8_LAYER_NORM if c["kind"] == "layer" else f8.F8_RMS_NORM
        if op == "norm_fwd":
            y, mean, rstd = f8.f8_norm_fwd(s["x"], s["w"], s["b"], kind=kind, eps=NORM_EPS, **s["out"])
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = f8.f8_norm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], kind=kind, **s["out"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "logprobs":
        logp, entropy, lse, ids, top = f8.f8_token_logprobs(s["logits"], s["tokens"], top_k=c["k"],
                                                            temperature=c["temperature"], **s["out"])
        return {"logp": logp, "entropy": entropy, "lse": lse, "top_ids": ids, "top_logp": top}
    if op == "logprobs_bwd":
        return {"dlogits": f8.f8_token_logprobs_bwd(s["logits"], s["tokens"], s["lse"], s["entropy"], s["dlogp"],
                                                    s["dentropy"], temperature=c["temperature"], dlogits=s["dlogits"])}
    kw = dict(temperature=c["temperature"], tail=c["tail"])
    if op == "distill_fwd":
        loss, lse, rest = f8.f8_distill_fwd(s["logits"], s["ids"], s["values"], loss=s["loss"], lse=s["lse"],
                                            rest=s["rest"], **kw)
        return {"loss": loss, "lse": lse, "rest": rest}
    if op == "distill_bwd":
        return {"dlogits": f8.f8_distill_bwd(s["logits"], s["ids"], s["values"], s["lse"], s["rest"], s["dloss"],
                                             dlogits=s["dlogits"], **kw)}
    loss, dlogits = f8.f8_distill_fwd_bwd(s["logits"], s["ids"], s["values"], s["dloss"], loss=s["loss"],
                                          dlogits=s["dlogits"], **kw)
    return {"loss": loss, "dlogits": dlogits}


def _softmax(z):
    """(max, exp(z - max), sum, log-sum-exp) by row."""
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    t = e.sum(1, keepdim=True)
    return e, t, (m + torch.log(t)).squeeze(1)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        x, w = s["x"].float(), s["w"].float()
        mean = x.mean(1, keepdim=True) if s["b"] is not None else None
        d = x - mean if mean is not None else x
        rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + NORM_EPS)
        y = d * rstd * w
        if s["b"] is not None:
            y = y + s["b"].float()
        return {"y": y.to(s["x"].dtype), "mean": None if mean is None else mean.squeeze(1), "rstd": rstd.squeeze(1)}
    if op == "norm_bwd":
        x, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
        rstd = s["rstd"][:, None]
        layer = s["mean"] is not None
        xhat = (x - s["mean"][:, None] if layer else x) * rstd
        g = dy * w
        dx = g - xhat * (g * xhat).mean(1, keepdim=True)
        if layer:
            dx = dx - g.mean(1, keepdim=True)
        dt = s["x"].dtype
        return {"dx": (dx * rstd).to(dt), "dw": (dy * xhat).sum(0).to(dt), "db": dy.sum(0).to(dt) if layer else None}
    return _plain_logits(s)


def _plain_logits(s):
    c = s["case"]
    op, k, vocab, tau = c["op"], c["k"], c["vocab"], c["temperature"]
    raw = s["logits"].float()
    z = raw / tau
    if op == "logprobs":
        tokens = s["tokens"]
        skip = tokens < 0
        e, t, lse = _softmax(z)
        p = e / t
        ent = lse - torch.where(p > 0, p * z, torch.zeros_like(p)).sum(1)
        logp = z.gather(1, tokens.clamp(min=0)[:, None]).squeeze(1) - lse
        out = {"logp": logp, "entropy": ent, "lse": lse}
        out = {n: torch.where(skip, torch.zeros_like(v), v) for n, v in out.items()}
        if not k:
            return out | {"top_ids": None, "top_logp": None}
        # one whole number for each value and place: larger values first, then lower places
        bits = (raw + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits)
        key = order * (1 << 32) + (vocab - 1 - torch.arange(vocab, device="cuda"))
        ids = vocab - 1 - (torch.topk(key, k, dim=1).values & 0xFFFFFFFF)
        top = z.gather(1, ids) - lse[:, None]
        out["top_ids"] = torch.where(skip[:, None], torch.full_like(ids, -1), ids).to(torch.int32)
        out["top_logp"] = torch.where(skip[:, None], torch.full_like(top, NEG_INF), top)
        return out
    width = s["full"].shape[1]
    if op == "logprobs_bwd":
        tokens, lse = s["tokens"], s["lse"][:, None]
        skip = (tokens < 0)[:, None]
        logp = z - lse
        p = torch.exp(logp)
        g = -s["dlogp"][:, None] * p
        g = g - s["dentropy"][:, None] * torch.where(p > 0, p * (logp + s["entropy"][:, None]), torch.zeros_like(p))
        at = tokens.clamp(min=0)[:, None]
        g.scatter_add_(1, at, torch.where(skip, torch.zeros_like(lse), s["dlogp"][:, None]))
        g = torch.where(skip, torch.zeros_like(g), g / tau)
        return {"dlogits": torch.nn.functional.pad(g, (0, width - vocab)).to(s["full"].dtype)}
    ids, values = s["ids"], s["values"]
    empty = ids < 0
    at = ids.clamp(min=0).long()
    live = (~empty).any(1)
    values = torch.where(empty, torch.full_like(values, NEG_INF), values)
    if c["tail"]:
        q = torch.exp(values)
        logq = values
    else:
        v = values / tau
        e, t, lse_q = _softmax(torch.where(live[:, None], v, torch.zeros_like(v)))
        q = torch.where(live[:, None], e / t, torch.zeros_like(e))
        logq = v - lse_q[:, None]
    out = {}
    if op == "distill_bwd":
        lse = s["lse"]
        p = torch.exp(z - lse[:, None])
        rest = s["rest"] if c["tail"] else None
    else:
        e, t, lse = _softmax(z)
        p = e / t
        if c["tail"]:
            outside = torch.cat((p, torch.zeros_like(p[:, :1])), 1)
            outside.scatter_(1, torch.where(empty, torch.full_like(at, vocab), at), 0.0)
            rest = outside.sum(1)
        logp = z.gather(1, at) - lse[:, None]
        loss = torch.where(empty, torch.zeros_like(q), q * (logq - logp)).sum(1)
        if c["tail"]:
            left = (1.0 - q.sum(1)).clamp(min=0.0)
            left = torch.where(rest > 0, left, torch.zeros_like(left))
            loss = loss + torch.where(left > 0, left * (torch.log(left) - torch.log(rest)), torch.zeros_like(left))
        zero = torch.zeros_like(loss)
        out["loss"] = torch.where(live, loss, zero)
        if op == "distill_fwd":
            out["lse"] = torch.where(live, lse, zero)
            out["rest"] = torch.where(live, rest, zero) if c["tail"] else None
            return out
    if c["tail"]:
        left = (1.0 - q.sum(1)).clamp(min=0.0)
        ratio = torch.where(rest > 0, left / rest, torch.zeros_like(left))
        total = q.sum(1) + torch.where(rest > 0, left, torch.zeros_like(left))
        inside = p.gather(1, at) * total[:, None] - q
        g = p * (total - ratio)[:, None]
    else:
        total = torch.where(live, torch.ones_like(lse), torch.zeros_like(lse))
        inside = p.gather(1, at) * total[:, None] - q
        g = p * total[:, None]
    g = torch.cat((g, torch.zeros_like(g[:, :1])), 1)
    g = g.scatter(1, torch.where(empty, torch.full_like(at, vocab), at), inside)[:, :vocab]
    scale = s["dloss"] / tau
    g = torch.where((scale == 0)[:, None] | ~live[:, None], torch.zeros_like(g), g * scale[:, None])
    out["dlogits"] = torch.nn.functional.pad(g, (0, width - vocab)).to(s["full"].dtype)
    return out


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """What the definitions give in 64 bits, row by row of the definition and not of the plain form's steps."""
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        x, w = s["x"].double(), s["w"].double()
        n = case["cols"]
        mu = x.sum(1, keepdim=True) / n if case["kind"] == "layer" else torch.zeros_like(x[:, :1])
        if op == "norm_fwd":
            var = ((x - mu) ** 2).sum(1, keepdim=True) / n
            r = 1.0 / torch.sqrt(var + NORM_EPS)
            y = (x - mu) * r * w + (s["b"].double() if s["b"] is not None else 0.0)
            return {"y": y, "mean": mu[:, 0] if case["kind"] == "layer" else None, "rstd": r[:, 0]}
        r = s["rstd"].double()[:, None]
        if case["kind"] == "layer":
            mu = s["mean"].double()[:, None]
        xh = (x - mu) * r
        dy = s["dy"].double()
        a = (dy * w * xh).sum(1, keepdim=True) / n
        m = (dy * w).sum(1, keepdim=True) / n if case["kind"] == "layer" else 0.0
        return {"dx": r * (dy * w - m - xh * a), "dw": (dy * xh).sum(0),
                "db": dy.sum(0) if case["kind"] == "layer" else None}
    return _exact_logits(case, s)


def _exact_logits(case, s):
    op, vocab, tau, k = case["op"], case["vocab"], case["temperature"], case["k"]
    u = s["logits"].double() / tau
    width = s["full"].shape[1]
    if op == "logprobs":
        tok = s["tokens"]
        keep = (tok >= 0).double()
        dead = tok < 0
        lse = torch.logsumexp(u, 1)
        lp = u - lse[:, None]
        p = lp.exp()
        ent = -(p * lp.clamp(min=-1e300)).sum(1)
        at = lp[torch.arange(len(tok), device="cuda"), tok.clamp(min=0)]
        out = {"logp": at.masked_fill(dead, 0.0), "entropy": ent * keep, "lse": lse * keep, "top_ids": None, "top_logp": None}
        if k:
            out["top_logp"] = lp.topk(k, dim=1).values.masked_fill(dead[:, None], NEG_INF)
        return out
    if op == "logprobs_bwd":
        tok = s["tokens"]
        lp = u - s["lse"].double()[:, None]
        p = lp.exp()
        hot = torch.zeros_like(p)
        hot[torch.arange(len(tok), device="cuda"), tok.clamp(min=0)] = 1.0
        surprise = torch.where(p > 0, lp, torch.zeros_like(lp)) + s["entropy"].double()[:, None]
        d = s["dlogp"].double()[:, None] * (hot - p) - s["dentropy"].double()[:, None] * p * surprise
        d = (d / tau).masked_fill((tok < 0)[:, None], 0.0)
        return {"dlogits": torch.cat((d, d.new_zeros((d.shape[0], width - vocab))), 1)}
    ids = s["ids"].long()
    have = ids >= 0
    live = have.any(1)
    t = s["values"].double().masked_fill(~have, NEG_INF)
    if not case["tail"]:
        t = t / tau
        t = t - torch.logsumexp(torch.where(live[:, None], t, torch.zeros_like(t)), 1, keepdim=True)
    # the teacher's distribution laid over the vocabulary, with one place after it for what has no id
    Q = u.new_zeros((u.shape[0], vocab + 1)).scatter_add_(1, torch.where(have, ids, vocab), t.exp())[:, :vocab]
    S = u.new_zeros((u.shape[0], vocab + 1)).scatter_(1, torch.where(have, ids, vocab), 1.0)[:, :vocab]
    lse = s["lse"].double() if op == "distill_bwd" else torch.logsumexp(u, 1)
    P = (u - lse[:, None]).exp()
    out = {}
    left = (1.0 - Q.sum(1)).clamp(min=0.0) if case["tail"] else torch.zeros_like(lse)
    if case["tail"]:
        rest = s["rest"].double() if op == "distill_bwd" else (P * (1.0 - S)).sum(1)
    else:
        rest = torch.ones_like(lse)
    left = left * (rest > 0)
    if op != "distill_bwd":
        kl = (Q * (torch.where(Q > 0, Q.log(), torch.zeros_like(Q)) - torch.where(Q > 0, u - lse[:, None], torch.zeros_like(Q)))).sum(1)
        kl = kl + torch.where(left > 0, left * (left.log() - rest.log()), torch.zeros_like(left))
        out["loss"] = kl.masked_fill(~live, 0.0)
    if op == "distill_fwd":
        out["lse"] = lse.masked_fill(~live, 0.0)
        out["rest"] = rest.masked_fill(~live, 0.0) if case["tail"] else None
        return out
    mass = Q.sum(1) + left
    share = torch.where(rest > 0, left / rest, torch.zeros_like(left)) if case["tail"] else torch.zeros_like(left)
    d = P * mass[:, None] - Q - (1.0 - S) * P * share[:, None]
    d = (d * (s["dloss"].double() / tau)[:, None]).masked_fill(~live[:, None], 0.0)
    out["dlogits"] = torch.cat((d, d.new_zeros((d.shape[0], width - vocab))), 1)
    return out
