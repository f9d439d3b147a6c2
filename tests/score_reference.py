"""The windowed attention with sinks whose scores are capped by a tanh or lowered by the
distance, in 64 bits from its definition, with the error that a bf16 kernel with fp32
statistics may make of it (U, E and TINY as in sink_reference).

Scores.  A product is off by d E of the sum of its terms' magnitudes S.  A cap c adds
2^-20 c (r = 1 / (1 + exp(2x/c)) and c - 2 c r in fp32, exp2 and the reciprocal off by
2^-22 and 2^-23 of their values: 2^-23 c times 3/4 for the exponent's three roundings,
since c z sech^2 z <= 0.45 c, 1 for exp2, 3 for 1 + E and the reciprocal, 2 for two
FMAs).  A bias b adds 8 E |b| (the slope's and the distance's roundings and those of the
sums), and where a block's 64 queries carry part of it, 8 E 64 |slope|.
With score errors e_s a weight p_s is off by p_s (e_s + sum p e), and lse by sum p e.
The cap's derivative 4 r (1 - r) is off by 2^-20 (r by 2^-21.4, 4 (1 - 2 r) times).
Gradients take delta_t = sum_s p_ts dP_ts, a sum in fp32 like the others.  For dq it stands
as the o given with delta~ = dO . o and a correction sigma times sum_s p_ts K_s, whose p are
rounded to bf16: U |sigma| sum p |K| more, sigma = scale (delta - delta~).
"""
import torch

from sink_reference import E, U, visible, within  # noqa: F401


def scores(q, k, qpos, kpos, cap, slopes, scale):
    """q [M, H, d], k [S, H, d] float64 -> scores, their errors, derivative by the product, [H, M, S]."""
    d = q.shape[-1]
    scale = d ** -0.5 if not scale else scale
    x = torch.einsum("mhd,shd->hms", q, k) * scale
    err = d * E * (torch.einsum("mhd,shd->hms", q.abs(), k.abs()) * scale + 1) + 2.0 ** -21
    turn = torch.ones_like(x)
    if cap:
        t = torch.tanh(x / cap)
        x, turn = cap * t, 1 - t * t
        err = err * turn + d * E + 2.0 ** -20 * cap + 2.0 ** -21
    if slopes is not None:
        b = slopes.double()[:, None, None] * (qpos[:, None] - kpos[None]).double()[None]
        x = x - b
        err = err + 8 * E * (b.abs() + 64 * slopes.double().abs()[:, None, None])
    return x, err, turn * scale


def rows(q, k, v, qpos, kpos, window, sinks, cap=0.0, slopes=None, scale=None):
    """As sink_reference.rows: o [M, H, d], lse [M, H] and their error bounds."""
    q, k, v = q.double(), k.double(), v.double()
    G = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    see = visible(qpos, kpos, window, sinks)
    s, err, _ = scores(q, k, qpos, kpos, cap, slopes, scale)
    s = s.masked_fill(~see, float("-inf"))
    empty = ~see.any(1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None].masked_fill(empty[None, :, None], 0.0))
    o = torch.einsum("hms,shd->mhd", p, v)
    av = torch.einsum("hms,shd->mhd", p, v.abs())
    el = (p * err).sum(-1) + len(kpos) * E                                  # [H, M]
    bo = U * (o.abs() + av) * 1.01 + 2 * (torch.einsum("hms,shd->mhd", p * err, v.abs()) + el.t()[..., None] * av)
    bl = 2 * el.t() + 4 * E * lse.t().abs().masked_fill(empty[:, None], 0)
    return o, lse.t(), bo, bl


def forward(q, k, v, window, sinks, cap=0.0, slopes=None, scale=None):
    pos = torch.arange(q.shape[1], device=q.device)
    out = [rows(q[b], k[b], v[b], pos, pos, window, sinks, cap, slopes, scale) for b in range(q.shape[0])]
    return [torch.stack(x) for x in zip(*out)]


def backward(q, k, v, o, lse, g, window, sinks, cap=0.0, slopes=None, scale=None):
    """Gradients for the given o and lse (the operator's inputs): (dq, dk, dv), bounds."""
    q, k, v, o, lse, g = (x.double() for x in (q, k, v, o, lse, g))
    B, L, H, d = q.shape
    Hkv = k.shape[2]
    G = H // Hkv
    pos = torch.arange(L, device=q.device)
    see = visible(pos, pos, window, sinks)
    res, bnd = [], []
    for b in range(B):
        kk, vv = k[b].repeat_interleave(G, 1), v[b].repeat_interleave(G, 1)
        s, err, turn = scores(q[b], kk, pos, pos, cap, slopes, scale)
        top = d ** -0.5 if not scale else scale                             # the greatest derivative
        p = torch.exp(s - lse[b].t()[..., None]).masked_fill(~see, 0)
        dp = torch.einsum("mhd,shd->hms", g[b], vv)
        da = torch.einsum("mhd,shd->hms", g[b].abs(), vv.abs())
        es = err + 4 * E * lse[b].t().abs()[..., None]
        dl = (p * dp).sum(-1, keepdim=True)
        dla = (g[b] * o[b]).abs().sum(-1).t()[..., None]
        err_dl = (p * (es * dp.abs() + d * E * (da + dla))).sum(-1, keepdim=True) + L * E * (p * (dp.abs() + dla)).sum(-1, keepdim=True)
        sigma = top * (dl - (g[b] * o[b]).sum(-1).t()[..., None]).abs()
        ds = turn * p * (dp - dl)
        err_p = p * (U + 2 * es)
        err_ds = ds.abs() * (U + 2 * es) * 1.01 + top * p * (d * E * (da + dla) * 2 + err_dl)
        if cap:
            err_ds = err_ds + 2.0 ** -20 * top * p * (dp - dl).abs()

        def fold(x):
            return x.view(L, Hkv, G, d).sum(2)
        dq = torch.einsum("hms,shd->mhd", ds, kk)
        dk = fold(torch.einsum("hms,mhd->shd", ds, q[b]))
        dv = fold(torch.einsum("hms,mhd->shd", p, g[b]))
        n = G * L * E                                                       # sums of up to G L terms in fp32
        bq = torch.einsum("hms,shd->mhd", err_ds + n * ds.abs() + (U * 1.01 + n) * sigma * p, kk.abs())
        bk = fold(torch.einsum("hms,mhd->shd", err_ds + n * ds.abs(), q[b].abs()))
        bv = fold(torch.einsum("hms,mhd->shd", err_p + n * p, g[b].abs()))
        res.append((dq, dk, dv))
        bnd.append((bq + U * dq.abs() * 1.01, bk + U * dk.abs() * 1.01, bv + U * dv.abs() * 1.01))
    return [torch.stack(x) for x in zip(*res)], [torch.stack(x) for x in zip(*bnd)]
