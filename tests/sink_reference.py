"""The windowed attention with sinks in 64 bits, from its definition, with the error
that a bf16 kernel with fp32 statistics may make of it.

Bounds, per element.  u = 2^-8 is the rounding of a value to bf16, e = 2^-24 to
fp32.  A kernel rounds the (unnormalised) weights to bf16 once before the
product with V, and the result once:
    |o - o'|   <= u |o| + u sum_s p_s |v_s|
Scores are sums of d products in fp32 (relative error d e of the sum of their
magnitudes S), so weights are off by about es = d e max S besides; the exponent
function adds 2^-21.  Gradients: ds and p are rounded to bf16 once, the result
once, dp is a sum of d products.  Weights below the smallest normal number,
2^-126, may be flushed to zero: n of them take at most n 2^-126 max |x| from a
sum, which TINY covers for n max |x| < 2^26.
"""
import torch

U, E = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -100


def visible(qpos, kpos, window, sinks):
    """[M, S] truth values; window 0: no window."""
    q, k = qpos[:, None], kpos[None, :]
    see = (k <= q) & (q >= 0)
    if window:
        see &= (k > q - window) | (k < sinks)
    return see


def rows(q, k, v, qpos, kpos, window, sinks, scale=None):
    """q [M, H, d] at positions qpos, k, v [S, Hkv, d] at kpos, any float type.  Returns
    o [M, H, d], lse [M, H] and their error bounds, float64."""
    q, k, v = q.double(), k.double(), v.double()
    M, H, d = q.shape
    G = H // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    scale = d ** -0.5 if not scale else scale
    see = visible(qpos, kpos, window, sinks)
    s = torch.einsum("mhd,shd->hms", q, k) * scale
    sa = torch.einsum("mhd,shd->hms", q.abs(), k.abs()) * scale
    s = s.masked_fill(~see, float("-inf"))
    empty = ~see.any(1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None].masked_fill(empty[None, :, None], 0.0))
    o = torch.einsum("hms,shd->mhd", p, v)
    es = (d * E * (sa.masked_fill(~see, 0).amax(-1) + 1) + len(kpos) * E + 2.0 ** -21)     # [H, M]
    av = torch.einsum("hms,shd->mhd", p, v.abs())
    bo = U * (o.abs() + av) * 1.01 + 2 * es.t()[..., None] * av
    bl = es.t() + 4 * E * lse.t().abs().masked_fill(empty[:, None], 0)
    return o, lse.t(), bo, bl


def forward(q, k, v, window, sinks, scale=None):
    """[B, L, H, d] -> o, lse, bounds."""
    pos = torch.arange(q.shape[1], device=q.device)
    out = [rows(q[b], k[b], v[b], pos, pos, window, sinks, scale) for b in range(q.shape[0])]
    return [torch.stack(x) for x in zip(*out)]


def backward(q, k, v, o, lse, g, window, sinks, scale=None):
    """Gradients for the given o and lse (the operator's inputs): (dq, dk, dv), bounds."""
    q, k, v, o, lse, g = (x.double() for x in (q, k, v, o, lse, g))
    B, L, H, d = q.shape
    Hkv = k.shape[2]
    G = H // Hkv
    scale = d ** -0.5 if not scale else scale
    pos = torch.arange(L, device=q.device)
    see = visible(pos, pos, window, sinks)
    res, bnd = [], []
    for b in range(B):
        kk, vv = k[b].repeat_interleave(G, 1), v[b].repeat_interleave(G, 1)
        s = torch.einsum("mhd,shd->hms", q[b], kk) * scale
        sa = torch.einsum("mhd,shd->hms", q[b].abs(), kk.abs()) * scale
        p = torch.exp(s - lse[b].t()[..., None]).masked_fill(~see, 0)
        dp = torch.einsum("mhd,shd->hms", g[b], vv)
        da = torch.einsum("mhd,shd->hms", g[b].abs(), vv.abs())
        dl = (g[b] * o[b]).sum(-1).t()[..., None]
        dla = (g[b] * o[b]).abs().sum(-1).t()[..., None]
        ds = scale * p * (dp - dl)
        # p is off by es relative; dp and delta by d e of their magnitudes
        es = d * E * (sa + 1) + 4 * E * lse[b].t().abs()[..., None] + 2.0 ** -21
        err_p = p * (U + 2 * es)
        err_ds = ds.abs() * (U + 2 * es) * 1.01 + scale * p * d * E * (da + dla) * 2

        def fold(x):
            return x.view(L, Hkv, G, d).sum(2)
        dq = torch.einsum("hms,shd->mhd", ds, kk)
        dk = fold(torch.einsum("hms,mhd->shd", ds, q[b]))
        dv = fold(torch.einsum("hms,mhd->shd", p, g[b]))
        bq = torch.einsum("hms,shd->mhd", err_ds, kk.abs())
        bk = fold(torch.einsum("hms,mhd->shd", err_ds, q[b].abs()))
        bv = fold(torch.einsum("hms,mhd->shd", err_p, g[b].abs()))
        # accumulation in fp32 over up to G L terms, as a sum of magnitudes
        n = G * L * E
        bq = bq + n * torch.einsum("hms,shd->mhd", ds.abs(), kk.abs())
        bk = bk + n * fold(torch.einsum("hms,mhd->shd", ds.abs(), q[b].abs()))
        bv = bv + n * fold(torch.einsum("hms,mhd->shd", p, g[b].abs()))
        res.append((dq, dk, dv))
        bnd.append((bq + U * dq.abs() * 1.01, bk + U * dk.abs() * 1.01, bv + U * dv.abs() * 1.01))
    return [torch.stack(x) for x in zip(*res)], [torch.stack(x) for x in zip(*bnd)]


def within(name, got, want, bound):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    ninf = torch.isneginf(want)
    assert torch.equal(torch.isneginf(got), ninf), "%s: -inf in the wrong places" % name
    got, want, bound = got[~ninf], want[~ninf], bound[~ninf]
    assert torch.isfinite(got).all(), "%s has non-finite values" % name
    over = (got - want).abs() - bound - TINY
    if got.numel() and float(over.max()) > 0:
        i = int(over.argmax())
        raise AssertionError("%s: %d of %d elements over their bound; worst got %.8g want %.8g bound %.3g"
                             % (name, int((over > 0).sum()), got.numel(), got[i], want[i], bound[i]))
