"""The norm, the token log probabilities and the distillation loss from their
definitions in 64 bits, and how far fp32 arithmetic with one final rounding may
be from them.

The bounds count roundings: u = 2^-24 is fp32's unit roundoff, and a result
formed in n fp32 steps from terms of total magnitude A is within n u A.  Sums
over a row run over at most 16 terms in a thread's chain (4 chains of them on
long rows, whose partial sums stay of one sign) and then over a tree of at most
13 levels; 2^x and ln are within 2 ulp.  K = 64 covers the steps of any one
result.  A bf16 output adds half a unit in its last place."""
import numpy as np
import torch

U = 2.0 ** -24
K = 64.0
TINY = 1e-37       # below fp32's normal range results may be flushed


def ulp(ref: torch.Tensor, dtype) -> torch.Tensor:
    """The spacing of dtype's values at ref (bf16: 8 significant bits, fp32: 24)."""
    bits = 7 if dtype == torch.bfloat16 else 23
    a = ref.abs().clamp(min=2.0 ** -126)
    return torch.exp2(torch.floor(torch.log2(a)) - bits)


def rounding(ref: torch.Tensor, dtype) -> torch.Tensor:
    """Half a unit in the last place of the stored type; a value next to a
    power of two may round on the wider side (1 %)."""
    return 0.505 * ulp(ref, dtype)


def check(got: torch.Tensor, ref: torch.Tensor, bound: torch.Tensor, what: str) -> None:
    g = got.double()
    # what lies past the range of the stored type is infinite in it
    big = float(torch.finfo(got.dtype).max)
    ref = torch.where(ref.abs() > big, torch.sign(ref) * float("inf"), ref)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(g[inf], ref[inf]) and not torch.isinf(g[~inf]).any(), f"{what}: infinities"
    ok = ~(nan | inf)
    err = (g - ref).abs()[ok]
    lim = (bound.expand_as(ref))[ok] + TINY
    if err.numel():
        worst = (err / lim).max().item()
        assert worst <= 1.0, f"{what}: {worst:.3g} times the bound (error {err.max().item():.3g})"


# ---------------------------------------------------------------- norm
def norm_fwd(x, w, b, rms, eps):
    """y, mean, rstd and the bounds of y, mean and rstd."""
    x, w = x.double(), w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    mu = torch.zeros_like(x[:, :1]) if rms else x.mean(1, keepdim=True)
    d = x - mu
    var = d.square().mean(1, keepdim=True)
    r = (var + eps).rsqrt()
    y = d * r * w + b
    size = x.abs().mean(1, keepdim=True)
    # an error of the mean shifts every difference; of the differences, r
    dmu = K * U * size * (0.0 if rms else 1.0)
    reach = x.abs() + size
    dr = r * K * U * (1.0 + r * r * d.abs().mean(1, keepdim=True) * size * (0.0 if rms else 1.0)) \
        + r ** 3 * dmu ** 2
    by = r * w.abs() * K * U * reach + d.abs() * w.abs() * dr + K * U * b.abs()
    return y, mu.squeeze(1), r.squeeze(1), by, dmu.squeeze(1), dr.squeeze(1)


def norm_bwd(dy, x, w, mean, rstd, rms):
    """dx, dw, db and their bounds, for the given fp32 statistics."""
    x, dy, w = x.double(), dy.double(), w.double()
    C = x.shape[1]
    mu = torch.zeros_like(x[:, :1]) if rms else mean.double()[:, None]
    r = rstd.double()[:, None]
    xh = (x - mu) * r
    g = dy * w
    c1 = (g * xh).sum(1, keepdim=True) / C
    c2 = torch.zeros_like(c1) if rms else g.sum(1, keepdim=True) / C
    dx = r * (g - c2 - xh * c1)
    dw, db = (dy * xh).sum(0), dy.sum(0)
    big = (x.abs() + mu.abs()) * r          # xh before its cancellation
    a1 = (g.abs() * big).mean(1, keepdim=True)
    a2 = torch.zeros_like(a1) if rms else g.abs().mean(1, keepdim=True)
    bdx = K * U * r * (g.abs() + a2 + big * a1)
    # a column's sum runs through one chain per group of rows and a chain over
    # the partial rows: at most as many steps as rows
    n = K + min(x.shape[0], 4096)
    bdw, bdb = n * U * (dy.abs() * big).sum(0), n * U * dy.abs().sum(0)
    return dx, dw, db, bdx, bdw, bdb


# ---------------------------------------------------------------- logits
def token_logprobs(logits, tokens, T, top_k):
    """lse, logp, entropy, top ids and log probabilities, and bounds."""
    z = logits.double() / T
    lse = torch.logsumexp(z, 1)
    none = lse == float("-inf")
    # differences to the maximum: at the type's lowest value even 64 bits of
    # lse have no room for log V
    d = z - torch.where(none, torch.zeros_like(lse), z.amax(1))[:, None]
    e = d.exp()
    s = e.sum(1, keepdim=True)
    lp = d - s.log()
    ent = (s.log() - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1, keepdim=True) / s).squeeze(1)
    ent = torch.where(none, torch.zeros_like(ent), torch.where(torch.isnan(lse), lse, ent))
    lp = torch.where(none[:, None], torch.full_like(lp, float("-inf")), lp)
    m = torch.where(none, torch.zeros_like(lse), z.amax(1)).abs()
    spread = np.log(z.shape[1]) + 1.0
    b = K * U * (m + spread + lse.abs().nan_to_num(posinf=0.0, neginf=0.0))
    out = {"lse": lse, "entropy": ent, "b_lse": b, "b_entropy": K * U * (1 + spread) * spread + 0 * b}
    if tokens is not None:
        out["logp"] = lp.gather(1, tokens.clamp(min=0)[:, None]).squeeze(1)
        zt = z.gather(1, tokens.clamp(min=0)[:, None]).squeeze(1).abs()
        out["b_logp"] = b + K * U * zt.nan_to_num(posinf=0.0)
    if top_k:
        # larger values first, equal ones by ascending id
        ids = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :top_k]
        out["top_ids"] = ids
        out["top_logp"] = lp.gather(1, ids)
        out["b_top"] = b[:, None] + K * U * z.gather(1, ids).abs().nan_to_num(posinf=0.0)
    return out


def token_logprobs_bwd(logits, tokens, lse, entropy, dlogp, dentropy, T):
    z = logits.double() / T
    lp = z - lse.double()[:, None]
    p = lp.exp()
    a = torch.zeros_like(lse).double() if dlogp is None else dlogp.double()
    h = torch.zeros_like(a) if dentropy is None else dentropy.double()
    H = torch.zeros_like(a) if entropy is None else entropy.double()
    hot = torch.zeros_like(p)
    if tokens is not None:
        hot.scatter_(1, tokens.clamp(min=0)[:, None], 1.0)
    surprise = torch.where(p > 0, lp, torch.zeros_like(lp)) + H[:, None]
    g = (a[:, None] * (hot - p) - h[:, None] * p * surprise) / T
    # p's relative error: that of its exponent
    zz = torch.where(p > 0, z, torch.zeros_like(z)).abs() + lse.double().abs()[:, None]
    size = a.abs()[:, None] * p + h.abs()[:, None] * p * (torch.where(p > 0, lp, torch.zeros_like(lp)).abs() + H.abs()[:, None] + 1)
    bound = K * U * (size * (1 + zz) + a.abs()[:, None] * hot) / T
    if tokens is not None:
        dead = (tokens < 0)[:, None]
        g, bound = g.masked_fill(dead, 0.0), bound.masked_fill(dead, 0.0)
    return g, bound


def distill(logits, ids, values, T, tail, dloss):
    """loss, lse, rest, dlogits and the bounds of loss, rest and dlogits."""
    z = logits.double() / T
    R, V = z.shape
    have = (ids >= 0) & (values != float("-inf"))
    live = have.any(1)
    at = torch.where(have, ids.long(), torch.full_like(ids.long(), V))
    t = values.double().masked_fill(~have, float("-inf"))
    if tail:
        q = t.exp()
        logq = t
    else:
        t = t / T
        top = torch.where(live, t.amax(1), torch.zeros_like(t[:, 0]))[:, None]
        e = (t - top).exp()
        s = e.sum(1, keepdim=True).clamp(min=1e-300)
        q = torch.where(live[:, None], e / s, torch.zeros_like(e))
        logq = t - top - s.log()
    lse = torch.logsumexp(z, 1)
    none = lse == float("-inf")
    p = torch.where(none[:, None], torch.zeros_like(z), (z - lse[:, None]).exp())
    ext = torch.cat((p, torch.zeros_like(p[:, :1])), 1)
    inside = torch.zeros_like(ext).scatter_(1, at, 1.0)[:, :V]
    Q = torch.zeros_like(ext).scatter_add_(1, at, q)[:, :V]
    rest = (p * (1 - inside)).sum(1)
    left = torch.zeros_like(rest)
    if tail:
        left = torch.where(rest > 0, (1 - q.sum(1)).clamp(min=0.0), left)
    lp = torch.cat((z - lse[:, None], torch.zeros_like(z[:, :1])), 1).gather(1, at)
    lp = torch.where(none[:, None], torch.full_like(lp, float("-inf")), lp)
    used = have & (q > 0)
    zero = torch.zeros_like(q)
    loss = torch.where(used, q * (torch.where(used, logq, zero) - torch.where(used, lp, zero)), zero).sum(1)
    ratio = torch.zeros_like(rest)
    if tail:
        ok = (left > 0) & (rest > 0)
        one = torch.ones_like(rest)
        loss = loss + torch.where(ok, left * (torch.where(ok, left, one).log() - torch.where(ok, rest, one).log()), 0 * rest)
        ratio = torch.where(rest > 0, left / torch.where(rest > 0, rest, one), ratio)
    mass = q.sum(1) + left if tail else torch.ones_like(rest)
    dead = (~live | (dloss == 0) | none)[:, None]
    sc = dloss.double()[:, None] / T
    g = sc * (p * mass[:, None] - Q - (1 - inside) * p * ratio[:, None])
    g = g.masked_fill(dead, 0.0)
    # bounds
    zt = torch.where(z == float("-inf"), torch.zeros_like(z), z).abs()
    lsea = lse.abs().nan_to_num(posinf=0.0, neginf=0.0)
    qa = (q * (1 + torch.where(used, logq, zero).abs() + torch.where(used, lp, zero).abs().nan_to_num(posinf=0.0)
               + lsea[:, None] + t.abs().nan_to_num(posinf=0.0))).sum(1)
    # q_r = 1 - sum q carries the absolute error of the sum; the dense part of
    # the gradient its quotient by p_r
    dleft = K * U * (1 + (q * t.abs().nan_to_num(posinf=0.0)).sum(1))
    logs = 0 * rest
    if tail:
        one = torch.ones_like(rest)
        logs = torch.where((left > 0) & (rest > 0), 2 + torch.where(left > 0, left, one).log().abs()
                           + torch.where(rest > 0, rest, one).log().abs(), 2 * one)
    prel = K * U * (1 + zt + lsea[:, None])
    bloss = K * U * qa + (dleft * logs + K * U * (1 + lsea) * left if tail else 0 * rest)
    brest = rest * K * U * (2 + lsea + zt.amax(1))
    drat = torch.where(rest > 0, dleft / torch.where(rest > 0, rest, torch.ones_like(rest)), 0 * rest)
    qrel = K * U * (1 + t.abs().nan_to_num(posinf=0.0))
    dQ = torch.zeros_like(ext).scatter_add_(1, at, q * qrel)[:, :V]
    bg = sc.abs() * (prel * p * (mass[:, None] + ratio[:, None]) + dQ + p * (dleft if tail else 0 * rest)[:, None]
                     + (1 - inside) * p * (drat if tail else 0 * rest)[:, None])
    return {"loss": loss.masked_fill(~live, 0.0), "lse": lse.masked_fill(~live, 0.0),
            "rest": rest.masked_fill(~live, 0.0), "dlogits": g, "b_loss": bloss, "b_rest": brest,
            "b_lse": K * U * (1 + lsea + zt.amax(1) + np.log(V)), "b_dlogits": bg.masked_fill(dead, 0.0)}
