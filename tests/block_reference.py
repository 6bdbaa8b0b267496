"""What stands between a block's linears from its definitions in 64 bits, and how
far fp32 arithmetic with one final rounding may be from them.

The bounds count roundings as tests/ops_reference.py does: u = 2^-24, a result
formed in n fp32 steps from terms of total magnitude A is within n u A, and K
covers the steps of any one result.  Errors of intermediate values are carried to
the result by the magnitudes of its terms (the `_mag` values): each is the
definition with every term and factor replaced by its size."""
import math

import torch

from ops_reference import K, U

SQRT2PI = math.sqrt(2.0 * math.pi)
C, CK = math.sqrt(2.0 / math.pi), 0.044715
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")


# ---------------------------------------------------------------- activations
def act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "relu2":
        return torch.where(z < 0, torch.zeros_like(z), z) ** 2
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    return z * torch.sigmoid(2.0 * C * (z + CK * z ** 3))


def slope(name, z):
    """act'(z), and the size of its terms."""
    one = torch.ones_like(z)
    if name == "none":
        return one, one
    if name == "relu":
        s = torch.where(z > 0, one, 0 * one)
        return s, s
    if name == "relu2":
        s = torch.where(z > 0, 2 * z, 0 * one)
        return s, s
    if name == "gelu":
        phi, cdf = torch.exp(-0.5 * z * z) / SQRT2PI, 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return cdf + z * phi, cdf + z.abs() * phi
    v = z if name == "silu" else 2.0 * C * (z + CK * z ** 3)
    dv = one if name == "silu" else 2.0 * C * (1.0 + 3.0 * CK * z * z)
    p, q = torch.sigmoid(v), torch.sigmoid(-v)
    # 1 - p is formed by subtraction: an absolute error of u
    return p * (1.0 + z * dv * q), p * (1.0 + z.abs() * dv)


def act_steps(z):
    """Relative error of act and slope in units of 2^-23: 2^x and the reciprocal
    are within 2, the polynomial of Phi within 4, and the exponents, of up to 2.3 |z|
    (1 + z^2 / 22) or 0.73 z^2 bits with three roundings, add their absolute error."""
    return 16.0 + 4.0 * z * z


def gemm_act(a, b, inv, bias, name, residual):
    """z, y and their bounds before the final rounding; a, b the codes' values in 64
    bits.  The products are exact; each of the K additions may cut off 2^-23 of the
    running sum, which the sum of the terms' sizes bounds."""
    k = a.shape[1]
    z = (a @ b.t()) * inv
    bz = (a.abs() @ b.abs().t()) * inv * (k * 2.0 ** -23)
    if bias is not None:
        z = z + bias.double()
        bz = bz + bias.double().abs() * U
    bz = bz + 4 * U * z.abs()
    y = act(name, z)
    steep = torch.maximum(torch.full_like(z, 1.2), 2.0 * (z.abs() + bz)) if name == "relu2" else 1.2
    by = bz * steep + act_steps(z) * 2.0 ** -23 * y.abs()
    if residual is not None:
        y = y + residual.double()
        by = by + 2 * U * y.abs()
    return z, y, bz, by


def act_bwd(dy, z, name):
    """dz, dbias and their bounds."""
    dy, z = dy.double(), z.double()
    s, mag = slope(name, z)
    dz, bz = dy * s, dy.abs() * mag * act_steps(z) * 2.0 ** -23
    n = dy.shape[0]
    return dz, dz.sum(0), bz, bz.sum(0) + (K + n) * U * (dy.abs() * s.abs()).sum(0)


# ---------------------------------------------------------------- rotary positions
def rope(x, positions, freqs, scale, interleaved, inverse):
    """The rotated [batch, seq, heads, dim] and its bound: cosine and sine within 2^-22
    of the factor (their own error and that of an angle held to 2^-25 of half a turn),
    three operations."""
    x = x.double()
    half = freqs.shape[0]
    t = positions.double()[..., None] * freqs * (-1.0 if inverse else 1.0)
    cos, sin = scale * torch.cos(t)[..., None, :], scale * torch.sin(t)[..., None, :]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    p, q = (head[..., 0::2], head[..., 1::2]) if interleaved else (head[..., :half], head[..., half:])
    y1, y2 = p * cos - q * sin, q * cos + p * sin
    size = (p.abs() + q.abs()) * abs(scale)
    if interleaved:
        y, m = torch.stack((y1, y2), -1).flatten(-2), torch.stack((size, size), -1).flatten(-2)
    else:
        y, m = torch.cat((y1, y2), -1), torch.cat((size, size), -1)
    y, m = torch.cat((y, rest), -1), torch.cat((m * 2.0 ** -21, 0 * rest), -1)
    still = (positions < 0)[..., None, None]
    return torch.where(still, x, y), torch.where(still, torch.zeros_like(m), m)


# ---------------------------------------------------------------- residual stream
def _rows(gate, gate_rows, rows):
    return gate.double().reshape(-1, gate.shape[-1])[torch.arange(rows, device=gate.device) // gate_rows]


def _norm(x, bx, w, b, layer, eps):
    """y, mean, 1/deviation and their bounds, for x known within bx."""
    w = w.double()
    mu = x.mean(1, keepdim=True) if layer else torch.zeros_like(x[:, :1])
    bm = bx.mean(1, keepdim=True) + K * U * x.abs().mean(1, keepdim=True) if layer else torch.zeros_like(mu)
    d = x - mu
    bd = bx + bm + U * (x.abs() + mu.abs())
    var = d.square().mean(1, keepdim=True)
    r = (var + eps).rsqrt()
    # 1/deviation: half the relative error of var + eps
    rel = K * U + ((2 * d.abs() + bd) * bd).mean(1, keepdim=True) * r * r
    y = d * r * w
    by = (bd * r + d.abs() * r * rel) * w.abs() + 4 * U * y.abs()
    if b is not None:
        y = y + b.double()
        by = by + 2 * U * y.abs()
    return y, mu[:, 0], r[:, 0], by, bm[:, 0], (r * rel)[:, 0]


def residual_norm_fwd(a, r, w_pre, b_pre, w_post, b_post, gate, gate_rows, scale, layer, eps):
    """{name: (value, bound)} of r_out, y and the four statistics."""
    out = {}
    u = a.double()
    bu = torch.zeros_like(u)
    if w_post is not None:
        u, mu, s, bu, bm, bs = _norm(u, bu, w_post, b_post, layer, eps)
        out["mean_post"], out["rstd_post"] = (mu, bm), (s, bs)
    if gate is not None:
        g = _rows(gate, gate_rows, a.shape[0])
        u, bu = u * g, bu * g.abs() + 2 * U * (u * g).abs()
    x = scale * r.double() + u
    bx = bu + 2 * U * ((scale * r.double()).abs() + u.abs())
    out["r_out"] = (x, bx)
    y, mu, s, by, bm, bs = _norm(x, bx, w_pre, b_pre, layer, eps)
    out["y"], out["mean_pre"], out["rstd_pre"] = (y, by), (mu, bm), (s, bs)
    return out


def _slope(g, mag, x, mu, s, layer):
    """The gradient of a norm's input for that of its unscaled output, and its size."""
    e = (x - mu) * s
    size = e.abs() + (x.abs() + mu.abs()) * s
    d = g - e * (g * e).mean(1, keepdim=True)
    m = mag + size * (mag * size).mean(1, keepdim=True)
    if layer:
        d, m = d - g.mean(1, keepdim=True), m + mag.mean(1, keepdim=True)
    return s * d, s * m, e, size


def residual_norm_bwd(dy, dr_out, a, r_out, stats, w_pre, w_post, b_post, gate, gate_rows, scale, layer):
    """{name: (value, bound)} of every gradient."""
    rows = a.shape[0]
    st = stats.double()[:, :, None]
    zero = torch.zeros_like(st[0])
    dy, x, a = dy.double(), r_out.double(), a.double()
    steps, sums = 4 * K * U, (4 * K + rows) * U
    d, m, e, size = _slope(dy * w_pre.double(), (dy * w_pre.double()).abs(), x, st[2] if layer else zero,
                           st[3], layer)
    out = {"dw_pre": ((dy * e).sum(0), sums * (dy.abs() * size).sum(0)),
           "db_pre": (dy.sum(0), sums * dy.abs().sum(0))}
    if dr_out is not None:
        d, m = d + dr_out.double(), m + dr_out.double().abs()
    out["dr"] = (scale * d, steps * abs(scale) * m)
    g = _rows(gate, gate_rows, rows) if gate is not None else torch.ones_like(a[:, :1])
    u, um = a, a.abs()
    if w_post is not None:
        w1 = w_post.double()
        da, dm, e, size = _slope(d * g * w1, m * (g * w1).abs(), a, st[0] if layer else zero, st[1], layer)
        out["dw_post"] = ((d * g * e).sum(0), sums * (m * g.abs() * size).sum(0))
        out["db_post"] = ((d * g).sum(0), sums * (m * g.abs()).sum(0))
        u, um = e * w1, size * w1.abs()
        if b_post is not None:
            u, um = u + b_post.double(), um + b_post.double().abs()
    else:
        da, dm = d * g, m * g.abs()
    out["da"] = (da, steps * dm)
    if gate is not None:
        groups = -(-rows // gate_rows)
        at = torch.arange(rows, device=a.device) // gate_rows
        zero = torch.zeros((groups, a.shape[1]), dtype=torch.float64, device=a.device)
        out["dgate"] = (zero.index_add(0, at, d * u), sums * zero.index_add(0, at, m * um))
    return out
