"""What stands between the Float8 linears of a block: epilogues, residual norms and rotary positions.

What is measured, case by case: the Float8 matrix product whose epilogue adds a bias, applies an activation and adds a
residual, with the activation's backward pass and the bias's gradient; the residual stream's update by a block's output
(its norm, its gate, the stream's scale) together with the norm in front of the next block, forward and backward with
every parameter's gradient; and the rotation of queries and keys by their positions, forward and backward.

``run`` computes the plain form (elementary torch operations in 32 bits, angles in 64, rounded once) unless ``own`` is
set, and then makes the framework's calls on the same state.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")
EPS = 1e-5


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of eight sequences through the FFN's first linear: reading the weight's codes is all of it
        dict(name="gemm_act_decode", op="gemm_act", m=8, n=14336, k=4096, fmt="e4m3", act="silu", bias="bf16",
             residual=False, z=False),
        # the FFN's first linear in training at the block's 8192 tokens; the activation's input is kept for the backward pass
        dict(name="gemm_act_ffn", op="gemm_act", m=8192, n=14336, k=4096, fmt="e4m3", act="gelu_tanh", bias="bf16",
             residual=False, z=True),
        # its second linear, back onto the residual stream
        dict(name="gemm_act_down", op="gemm_act", m=8192, n=4096, k=14336, fmt="e4m3", act="none", bias="bf16",
             residual=True, z=False),
        # a ragged batch, an odd width, and a bias held in 32 bits
        dict(name="gemm_act_odd", op="gemm_act", m=1000, n=5003, k=2064, fmt="e5m2", act="gelu", bias="f32",
             residual=True, z=True),
        # the activation's backward pass at the FFN's width, with the bias's gradient
        dict(name="act_bwd_ffn", op="act_bwd", rows=8192, cols=14336, act="gelu_tanh", bias="bf16"),
        # a ragged one
        dict(name="act_bwd_odd", op="act_bwd", rows=1999, cols=5003, act="gelu", bias="f32"),
        # between two blocks while eight sequences decode one token each: one launch's latency
        dict(name="residual_norm_fwd_decode", op="residual_norm_fwd", kind="rms", dtype="bf16", stream="bf16", rows=8,
             cols=4096, post=True, gate="none", gate_rows=8, scale=1.0),
        # in training, with a gate for each of eight sequences
        dict(name="residual_norm_fwd_block", op="residual_norm_fwd", kind="layer", dtype="bf16", stream="bf16",
             rows=8192, cols=4096, post=True, gate="rows", gate_rows=1024, scale=1.0),
        # the backward pass, with the norms' and the gate's gradients
        dict(name="residual_norm_bwd_block", op="residual_norm_bwd", kind="rms", dtype="bf16", stream="bf16", rows=8192,
             cols=4096, post=True, gate="rows", gate_rows=8192, scale=1.0),
        # ragged sequences, a width that no vector divides, and a residual stream in 32 bits
        dict(name="residual_norm_bwd_odd", op="residual_norm_bwd", kind="layer", dtype="bf16", stream="f32", rows=1999,
             cols=5003, post=True, gate="rows", gate_rows=250, scale=0.5),
        # queries and keys of eight sequences that decode one token each, at far positions of a stretched context
        dict(name="rope_decode", op="rope", batch=8, seq=1, hq=32, hk=8, dim=128, rot=128, layout="half", dtype="bf16",
             inverse=False, far=True, packed=False, padded=0.0),
        # the gradient of the queries' and keys' columns of one packed projection, a part of each head rotated, rows padded
        dict(name="rope_bwd_packed", op="rope", batch=8, seq=1024, hq=32, hk=8, dim=128, rot=96, layout="interleaved",
             dtype="bf16", inverse=True, far=False, packed=True, padded=0.05),
    ]


OPS = ("gemm_act", "gemm_act", "act_bwd", "residual_norm_fwd", "residual_norm_bwd", "rope")
MOST_PRODUCTS = 8192 * 14336 * 4096
MOST_ELEMENTS = 8192 * 14336


def _spread(rng, lo, hi, near=128):
    """A whole number, its logarithm spread over [lo, hi]; a third are multiples of `near`, the others as they fall."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 1 / 3 and n >= near:
        n -= n % near
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(OPS)
    if op == "gemm_act":
        n = _spread(rng, 64, 16384)
        k = 16 * _spread(rng, 4, 1024, 8)
        m = _spread(rng, 1, max(1, min(16384, MOST_PRODUCTS // (n * k), MOST_ELEMENTS // n)))
        if rng.random() < 0.6:
            n += -n % 16
        return dict(op=op, m=m, n=n, k=k, fmt=rng.choice(("e4m3", "e4m3", "e5m2")), act=rng.choice(ACTS),
                    bias=rng.choice(("none", "bf16", "f32")), residual=rng.random() < 0.5, z=rng.random() < 0.5)
    if op == "act_bwd":
        cols = _spread(rng, 64, 28672)
        if rng.random() < 0.6:
            cols += -cols % 8
        return dict(op=op, rows=_spread(rng, 1, min(16384, MOST_ELEMENTS // cols)), cols=cols,
                    act=rng.choice(ACTS[1:]), bias=rng.choice(("none", "bf16", "f32")))
    if op == "rope":
        dim = rng.choice((64, 80, 96, 128, 128, 128, 192, 256))
        rot = rng.choice((dim, dim, dim // 2, 2 * (dim // 8)))
        heads = rng.choice((1, 1, 2, 4, 8))
        hq, hk = heads * rng.choice((1, 4, 5, 8)), heads
        tokens = _spread(rng, 1, min(32768, MOST_ELEMENTS // ((hq + 2 * hk) * dim * 2)))
        batch = rng.choice([b for b in (1, 2, 3, 8, 64) if b <= tokens])
        if rng.random() < 0.2:
            batch = tokens  # every sequence decodes one token
        return dict(op=op, batch=batch, seq=tokens // batch, hq=hq, hk=hk, dim=dim, rot=rot,
                    layout=rng.choice(("half", "interleaved")), dtype=rng.choice(("bf16", "bf16", "f32")),
                    inverse=rng.random() < 0.4, far=rng.random() < 0.4, packed=rng.random() < 0.4,
                    padded=rng.choice((0.0, 0.0, 0.1)))
    dtype, stream = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")))
    cols = _spread(rng, 64, 16384)
    if rng.random() < 0.6:
        cols += -cols % 8
    rows = _spread(rng, 1, min(16384, MOST_ELEMENTS // (4 * cols)))
    return dict(op=op, kind=rng.choice(("layer", "rms")), dtype=dtype, stream=stream, rows=rows, cols=cols,
                post=rng.random() < 0.7, gate=rng.choice(("none", "rows", "rows")),
                gate_rows=rng.choice((rows, rows, max(1, rows // 8), _spread(rng, 1, rows))),
                scale=rng.choice((1.0, 1.0, 0.5)))


def _size(name):
    return {"bf16": 2, "f32": 4, "none": 0}[name]


def _groups(case):
    return -(-case["rows"] // case["gate_rows"]) if case["gate"] == "rows" else 0


def work(case):
    """Each input read once and each output written once; the operations of the definition."""
    op = case["op"]
    if op == "gemm_act":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + n * _size(case["bias"]) + 2 * m * n * (1 + case["residual"] + case["z"]),
                "flops": 2 * m * n * k}
    if op == "act_bwd":
        e = case["rows"] * case["cols"]
        return {"bytes": 6 * e + case["cols"] * _size(case["bias"]), "flops": 12 * e}
    if op == "rope":
        heads = case["hq"] + case["hk"]
        tokens = case["batch"] * case["seq"]
        return {"bytes": 2 * tokens * heads * case["dim"] * _size(case["dtype"]) + 8 * tokens + 4 * case["rot"],
                "flops": 3 * tokens * heads * case["rot"]}
    rows, cols = case["rows"], case["cols"]
    e, x, r = rows * cols, _size(case["dtype"]), _size(case["stream"])
    params = (2 if case["kind"] == "layer" else 1) * (2 if case["post"] else 1)
    stats = 4 * rows * params
    gate = _groups(case) * cols * x
    if op == "residual_norm_fwd":
        return {"bytes": e * (2 * x + 2 * r) + params * cols * x + gate + stats, "flops": 16 * e}
    return {"bytes": e * (3 * x + 3 * r) + 2 * params * cols * x + 2 * gate + stats, "flops": 30 * e}


# ---------------------------------------------------------------- inputs
def _frequencies(rot, far):
    """Radians a position for each pair. `far`: a context stretched eightfold, slow pairs slowed down by it, fast ones
    kept, with a ramp between; cosines and sines then carry a factor."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if not far:
        return f.cuda(), 1.0
    turns = 8192.0 * f / (2.0 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return (f * keep + f / 8.0 * (1.0 - keep)).cuda(), 0.1 * math.log(8.0) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    op = case["op"]
    s = {"case": case}

    def rand(shape, std=1.0, dtype=torch.bfloat16, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    if op == "gemm_act":
        m, n, k = case["m"], case["n"], case["k"]
        for name, shape, std, fmt in (("a", (m, k), 1.0, case["fmt"]), ("b", (n, k), 1.3 / math.sqrt(k), "e4m3")):
            code, most = CODES[fmt]
            x = rand(shape, std).float()
            scale = (most / x.abs().amax()).reshape(1)
            s[name] = (x * scale).clamp_(-most, most).to(code).view(torch.uint8)
            s["scale_" + name] = scale
        s["bias"] = rand((n,), 0.5, TYPES[case["bias"]]) if case["bias"] != "none" else None
        s["residual"] = rand((m, n)) if case["residual"] else None
        s["y"] = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        s["z"] = torch.empty_like(s["y"]) if case["z"] else None
        return s
    if op == "act_bwd":
        shape = (case["rows"], case["cols"])
        s["z"] = rand(shape, 1.4)
        s["dy"] = rand(shape, 0.01)
        s["dz"] = torch.empty_like(s["z"])
        s["dbias"] = torch.empty(shape[1:], dtype=TYPES[case["bias"]], device="cuda") if case["bias"] != "none" else None
        return s
    if op == "rope":
        b, t, hq, hk, dim = case["batch"], case["seq"], case["hq"], case["hk"], case["dim"]
        dt = TYPES[case["dtype"]]
        s["freqs"], s["scale"] = _frequencies(case["rot"], case["far"])
        if case["packed"]:  # one projection's columns: queries, keys, values
            full = rand((b, t, hq + 2 * hk, dim), 1.0, dt)
            s["q"], s["k"] = full[:, :, :hq], full[:, :, hq:hq + hk]
        else:
            s["q"], s["k"] = rand((b, t, hq, dim), 1.0, dt), rand((b, t, hk, dim), 1.0, dt)
        first = torch.randint(0, 60000 if case["far"] else 3000, (b, 1), generator=gen, device="cuda")
        at = first + torch.arange(t, device="cuda")
        gone = torch.arange(t, device="cuda") >= t - int(case["padded"] * t)  # rows behind a sequence's end
        s["positions"] = torch.where(gone, torch.full_like(at, -1), at)
        s["q_out"] = torch.empty((b, t, hq, dim), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((b, t, hk, dim), dtype=dt, device="cuda")
        return s
    rows, cols = case["rows"], case["cols"]
    dt, st = TYPES[case["dtype"]], TYPES[case["stream"]]
    layer, post = case["kind"] == "layer", case["post"]
    spread = 0.5 + 2.0 * torch.rand((cols,), generator=gen, device="cuda")
    s["a"] = (torch.randn((rows, cols), generator=gen, device="cuda") * spread + 0.2).to(dt)
    s["r"] = rand((rows, cols), 2.0, st, 0.3)
    s["w_pre"] = rand((cols,), 0.2, dt, 1.0)
    s["b_pre"] = rand((cols,), 0.1, dt) if layer else None
    s["w_post"] = rand((cols,), 0.2, dt, 1.0) if post else None
    s["b_post"] = rand((cols,), 0.1, dt) if layer and post else None
    s["gate"] = rand((_groups(case), cols), 0.5, dt, 0.7) if case["gate"] == "rows" else None
    s["stats"] = torch.zeros((4, rows), device="cuda")
    if op == "residual_norm_fwd":
        s["out"] = {"r_out": torch.empty_like(s["r"]), "y": torch.empty_like(s["a"]), "stats": s["stats"]}
        return s
    # what the forward pass kept: the updated stream and the statistics
    r_out, _, s["stats"] = _forward(s)
    s["r_out"] = r_out.to(st)
    del s["r"]
    s["dy"] = rand((rows, cols), 0.01, dt)
    s["dr_out"] = rand((rows, cols), 0.01, st)
    like = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    s["out"] = {"da": like(s["a"]), "dr": like(s["r_out"]), "dw_pre": like(s["w_pre"]), "db_pre": like(s["b_pre"]),
                "dw_post": like(s["w_post"]), "db_post": like(s["b_post"]), "dgate": like(s["gate"])}
    return s


# ---------------------------------------------------------------- the two forms
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import float8_mixed_precision_gb300 as f8
    c = s["case"]
    op = c["op"]
    if op == "gemm_act":
        y, z = f8.f8_gemm_act(s["a"], s["b"], s["scale_a"], s["scale_b"], bias=s["bias"],
                              act=getattr(f8, "F8_ACT_" + c["act"].upper()), residual=s["residual"], y=s["y"], z=s["z"],
                              fmt_a=f8.F8_E5M2 if c["fmt"] == "e5m2" else f8.F8_E4M3)
        return {"y": y, "z": z}
    if op == "act_bwd":
        dz, dbias = f8.f8_act_bwd(s["dy"], s["z"], getattr(f8, "F8_ACT_" + c["act"].upper()), dz=s["dz"],
                                  dbias=s["dbias"], want_dbias=s["dbias"] is not None)
        return {"dz": dz, "dbias": dbias}
    if op == "rope":
        q, k = f8.f8_rope(s["q"], s["positions"], s["freqs"], k=s["k"],
                          layout=f8.F8_ROPE_HALF if c["layout"] == "half" else f8.F8_ROPE_INTERLEAVED,
                          scale=s["scale"], inverse=c["inverse"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    kw = dict(gate=s["gate"], gate_rows=c["gate_rows"] if s["gate"] is not None else None, scale=c["scale"],
              kind=f8.F8_LAYER_NORM if c["kind"] == "layer" else f8.F8_RMS_NORM)
    if op == "residual_norm_fwd":
        r_out, y, stats = f8.f8_residual_norm_fwd(s["a"], s["r"], s["w_pre"], b_pre=s["b_pre"], w_post=s["w_post"],
                                                  b_post=s["b_post"], eps=EPS, **kw, **s["out"])
        return {"r_out": r_out, "y": y} | _kept(c, stats)
    f8.f8_residual_norm_bwd(s["dy"], s["dr_out"], s["a"], s["r_out"], s["w_pre"], s["stats"], w_post=s["w_post"],
                            b_post=s["b_post"], **kw, **s["out"])
    return dict(s["out"])


def _kept(case, stats):
    """The statistics that a case has: those of the norm after a block and of the one in front of the next."""
    mean, post = case["kind"] == "layer", case["post"]
    return {"mean_post": stats[0] if mean and post else None, "rstd_post": stats[1] if post else None,
            "mean_pre": stats[2] if mean else None, "rstd_pre": stats[3]}


def _act(act, z):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "relu2":
        return torch.where(z < 0, torch.zeros_like(z), z * z)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    return z / (1.0 + torch.exp(-2.0 * u))


def _act_slope(act, z):
    if act == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), torch.ones_like(z))
    if act == "relu2":
        return torch.where(z <= 0, torch.zeros_like(z), 2.0 * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 / (1.0 + torch.exp(z))))
    if act == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    u = c * (z + 0.044715 * z * z * z)
    p = 1.0 / (1.0 + torch.exp(-2.0 * u))
    q = 1.0 / (1.0 + torch.exp(2.0 * u))
    return p + z * 2.0 * p * q * c * (1.0 + 3.0 * 0.044715 * z * z)


def _normed(x, w, b, layer):
    """(norm of the rows, mean, rstd)"""
    mean = x.mean(1, keepdim=True) if layer else None
    d = x - mean if layer else x
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    y = d * rstd * w.float()
    return y if b is None else y + b.float(), mean, rstd


def _by_row(s):
    """The gate's row for each row."""
    c = s["case"]
    return s["gate"].float()[torch.arange(c["rows"], device="cuda") // c["gate_rows"]]


def _forward(s):
    """(updated stream, its norm, statistics), in 32 bits."""
    c = s["case"]
    layer = c["kind"] == "layer"
    stats = torch.zeros((4, c["rows"]), device="cuda")
    u = s["a"].float()
    if s["w_post"] is not None:
        u, mean, rstd = _normed(u, s["w_post"], s["b_post"], layer)
        stats[1] = rstd[:, 0]
        if layer:
            stats[0] = mean[:, 0]
    if s["gate"] is not None:
        u = u * _by_row(s)
    r = s["r"].float() * c["scale"] + u
    y, mean, rstd = _normed(r, s["w_pre"], s["b_pre"], layer)
    stats[3] = rstd[:, 0]
    if layer:
        stats[2] = mean[:, 0]
    return r, y, stats


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "gemm_act":
        a = s["a"].view(CODES[c["fmt"]][0]).float()
        b = s["b"].view(CODES["e4m3"][0]).float()
        z = torch.matmul(a, b.t()) / (s["scale_a"] * s["scale_b"])
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(c["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(torch.bfloat16), "z": z.to(torch.bfloat16) if c["z"] else None}
    if op == "act_bwd":
        dz = s["dy"].float() * _act_slope(c["act"], s["z"].float())
        return {"dz": dz.to(torch.bfloat16),
                "dbias": None if s["dbias"] is None else dz.sum(0, dtype=torch.float64).to(s["dbias"].dtype)}
    if op == "rope":
        angle = s["positions"].double()[:, :, None] * s["freqs"]
        cos, sin = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
        if c["inverse"]:
            sin = -sin
        still = (s["positions"] < 0)[:, :, None, None]
        return {n: _rotated(s[n], cos[:, :, None], sin[:, :, None], still, c) for n in ("q", "k")}
    if op == "residual_norm_fwd":
        r, y, stats = _forward(s)
        return {"r_out": r.to(s["r"].dtype), "y": y.to(s["a"].dtype)} | _kept(c, stats)
    return _plain_backward(s)


def _rotated(x, cos, sin, still, c):
    rot = c["rot"]
    v = x.float()
    if c["layout"] == "half":
        x1, x2 = v[..., :rot // 2], v[..., rot // 2:rot]
        y = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin, v[..., rot:]), -1)
    else:
        x1, x2 = v[..., 0:rot:2], v[..., 1:rot:2]
        y = torch.cat((torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2), v[..., rot:]), -1)
    return torch.where(still, v, y).to(x.dtype)


def _norm_slope(g, xhat, rstd, layer):
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    return (d - g.mean(1, keepdim=True) if layer else d) * rstd


def _plain_backward(s):
    c = s["case"]
    layer = c["kind"] == "layer"
    dt, st = s["a"].dtype, s["r_out"].dtype
    dy, stats = s["dy"].float(), s["stats"]
    xhat = (s["r_out"].float() - stats[2][:, None] if layer else s["r_out"].float()) * stats[3][:, None]
    out = {"da": None, "dr": None, "dw_pre": (dy * xhat).sum(0).to(dt), "db_pre": dy.sum(0).to(dt) if layer else None,
           "dw_post": None, "db_post": None, "dgate": None}
    d = s["dr_out"].float() + _norm_slope(dy * s["w_pre"].float(), xhat, stats[3][:, None], layer)
    out["dr"] = (d * c["scale"]).to(st)
    u = s["a"].float()
    if c["post"]:
        xhat = (u - stats[0][:, None] if layer else u) * stats[1][:, None]
        u = xhat * s["w_post"].float()
        if layer:
            u = u + s["b_post"].float()
    du = d
    if s["gate"] is not None:
        group = torch.arange(c["rows"], device="cuda") // c["gate_rows"]
        out["dgate"] = torch.zeros_like(s["gate"], dtype=torch.float64).index_add_(0, group, (d * u).double()).to(dt)
        du = d * _by_row(s)
    if not c["post"]:
        out["da"] = du.to(dt)
        return out
    out["dw_post"] = (du * xhat).sum(0).to(dt)
    out["db_post"] = du.sum(0).to(dt) if layer else None
    out["da"] = _norm_slope(du * s["w_post"].float(), xhat, stats[1][:, None], layer).to(dt)
    return out


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """What the definitions give in 64 bits, written apart from the plain form's steps."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm_act":
        factor = 1.0 / (s["scale_a"].double() * s["scale_b"].double())
        # products of the codes' values are sums of at most 2^32 steps of 2^-25: 64 bits hold them
        z = (s["a"].view(CODES[case["fmt"]][0]).double() @ s["b"].view(CODES["e4m3"][0]).double().t()).mul_(factor)
        if s["bias"] is not None:
            z.add_(s["bias"].double())
        y = _exact_act(case["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, "z": z if case["z"] else None}
    if op == "act_bwd":
        z = s["z"].double().requires_grad_(True)
        dz, = torch.autograd.grad(_exact_act(case["act"], z), z, s["dy"].double())
        return {"dz": dz, "dbias": None if s["dbias"] is None else dz.sum(0)}
    if op == "rope":
        # a pair is a complex number, turned by exp(i angle)
        turn = torch.polar(torch.full((), s["scale"], dtype=torch.float64, device="cuda"),
                           torch.zeros((), dtype=torch.float64, device="cuda"))
        angle = s["positions"].double()[..., None] * s["freqs"] * (-1.0 if case["inverse"] else 1.0)
        turn = turn * torch.polar(torch.ones_like(angle), angle)
        turn = torch.where((s["positions"] < 0)[..., None], torch.ones_like(turn), turn)[:, :, None]
        return {n: _exact_rotated(s[n].double(), turn, case) for n in ("q", "k")}
    if op == "residual_norm_fwd":
        return _exact_forward(case, s)
    # the backward pass by definition: the derivative of <dr_out, r_out> + <dy, y>, with the statistics' own slopes
    # written out for the inputs that are given
    return _exact_backward(case, s)


def _exact_act(act, z):
    if act == "none":
        return z
    if act in ("relu", "relu2"):
        return torch.relu(z) if act == "relu" else torch.relu(z) ** 2
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))


def _exact_rotated(x, turn, case):
    rot = case["rot"]
    if case["layout"] == "half":
        p = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        head = torch.cat((p.real, p.imag), -1)
    else:
        head = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
    return torch.cat((head, x[..., rot:]), -1)


def _exact_rows(case):
    return torch.arange(case["rows"], device="cuda").div(case["gate_rows"], rounding_mode="floor")


def _exact_forward(case, s):
    layer = case["kind"] == "layer"
    n = case["cols"]

    def norm(x, w, b):
        mu = x.sum(1) / n if layer else torch.zeros_like(x[:, 0])
        rstd = 1.0 / torch.sqrt(((x - mu[:, None]) ** 2).sum(1) / n + EPS)
        y = torch.einsum("rc,r,c->rc", x - mu[:, None], rstd, w.double())
        return (y if b is None else y + b.double()), mu, rstd

    u = s["a"].double()
    out = {"mean_post": None, "rstd_post": None}
    if case["post"]:
        u, mu, out["rstd_post"] = norm(u, s["w_post"], s["b_post"])
        out["mean_post"] = mu if layer else None
    if s["gate"] is not None:
        u = s["gate"].double().index_select(0, _exact_rows(case)) * u
    r = case["scale"] * s["r"].double() + u
    y, mu, rstd = norm(r, s["w_pre"], s["b_pre"])
    return {"r_out": r, "y": y} | out | {"mean_pre": mu if layer else None, "rstd_pre": rstd}


def _exact_backward(case, s):
    layer = case["kind"] == "layer"
    n = case["cols"]
    stats = s["stats"].double()

    def slope(g, x, mu, rstd, w):
        """The derivative to x of <g, norm(x)>, from its Jacobian's three terms."""
        e = (x - mu[:, None]) * rstd[:, None]
        h = g * w.double()
        along = torch.einsum("rc,rc->r", h, e) / n
        level = h.sum(1) / n if layer else torch.zeros_like(along)
        return rstd[:, None] * (h - level[:, None] - along[:, None] * e), e

    dy = s["dy"].double()
    d, e = slope(dy, s["r_out"].double(), stats[2], stats[3], s["w_pre"])
    out = {"dw_pre": torch.einsum("rc,rc->c", dy, e), "db_pre": dy.sum(0) if layer else None}
    d = d + s["dr_out"].double()
    out["dr"] = case["scale"] * d
    a = s["a"].double()
    rows = _exact_rows(case)
    g = s["gate"].double().index_select(0, rows) if s["gate"] is not None else torch.ones_like(a[:1])
    if case["post"]:
        da, e = slope(d * g, a, stats[0], stats[1], s["w_post"])
        u = e * s["w_post"].double() + (s["b_post"].double() if layer else 0.0)
        out["dw_post"] = (d * g * e).sum(0)
        out["db_post"] = (d * g).sum(0) if layer else None
    else:
        da, u = d * g, a
        out["dw_post"] = out["db_post"] = None
    out["da"] = da
    out["dgate"] = None
    if s["gate"] is not None:
        out["dgate"] = torch.stack([(d * u)[rows == i].sum(0) for i in range(len(s["gate"]))]) if len(s["gate"]) <= 64 else \
            torch.zeros_like(s["gate"], dtype=torch.float64).index_add_(0, rows, d * u)
    return {k: out[k] for k in ("da", "dr", "dw_pre", "db_pre", "dw_post", "db_post", "dgate")}
