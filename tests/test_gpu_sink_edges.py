"""Calls of the windowed attention with sinks and of its paged cache that stand at the edge of
what their documentation allows."""
import pytest
import torch

from retrieval_sparse_attention_gb300 import api

import sink_reference as ref

pytestmark = pytest.mark.gpu

BAD_INDEX = 6


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_append_without_query_heads():
    g = torch.Generator().manual_seed(1)
    kn, vn = (torch.randn(5, 2, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    kc, vc = (torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p = api.make_paged_params(B=2, total_q=5, Hkv=2, d=64, page=16, n_pages=4, table_width=2)
    p.H = 0
    api.gca_paged_append(p, kn, vn, ints(0, 3, 5), ints(17, 2), ints(2, 1, 3, 0).view(2, 2), kc, vc)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    for c, n in ((kc, kn), (vc, vn)):
        assert torch.equal(torch.cat([c[2, 14:], c[1, :1], c[3, :2]]), n)
        assert int((c.abs().sum((-1, -2)) > 0).sum()) == 5


# rows of q that are not finite, in units left whole and in units that are cut and joined
@pytest.mark.parametrize("L,H,Hkv,d,window,sinks,launches", [(300, 4, 2, 64, 90, 4, 1), (700, 3, 3, 128, 40, 130, 1),
                                                             (6000, 2, 1, 64, 6000, 0, 2), (3300, 12, 12, 64, 1500, 4, 1)])
def test_a_query_that_is_not_finite_gets_nan_and_stays_alone(L, H, Hkv, d, window, sinks, launches):
    g = torch.Generator().manual_seed(L)
    q, k, v = (torch.randn(1, L, h, d, generator=g).to(torch.bfloat16) for h in (H, Hkv, Hkv))
    k[..., 0] = -k[..., 0].abs() - 0.5           # (an infinite q[0] makes every score -inf, or +inf)
    nan, inf = float("nan"), float("inf")
    bad = [(0, 0, nan), (1, H - 1, inf), (L // 2, 0, inf), (L // 2 + 1, 1, -inf), (L // 3, 1, nan), (L - 1, 0, nan)]
    qc, kc, vc = (x.cuda() for x in (q, k, v))
    o, lse = api.swa_sink_fwd(qc, kc, vc, window=window, sinks=sinks)
    for t, h, x in bad:
        qc[0, t, h, 0] = x
    ob, lseb = api.swa_sink_fwd(qc, kc, vc, window=window, sinks=sinks)
    assert api.gca_last_launch_count() == launches
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    for t, h, x in bad:
        assert torch.isnan(ob[0, t, h]).all() and torch.isnan(lseb[0, t, h]), (t, h, x)
        ob[0, t, h], lseb[0, t, h] = o[0, t, h], lse[0, t, h]
    assert torch.equal(ob, o) and torch.equal(lseb, lse)


@pytest.mark.parametrize("n,kv", [(5, 3), (3, 3000)])
def test_queries_over_the_cache_that_are_not_finite(n, kv):
    g = torch.Generator().manual_seed(kv)
    page, pages = 16, -(-kv // 16)
    kc, vc = (torch.randn(pages, page, 1, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    kc[..., 0] = -kc[..., 0].abs() - 0.5
    q = torch.randn(n, 2, 64, generator=g).to(torch.bfloat16).cuda()
    args = (kc, vc, torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1), ints(0, n), ints(kv))
    o, lse = api.paged_attn(q, *args, with_lse=True)
    qb = q.clone()
    qb[0, 0, 3], qb[1, 1, 0], qb[n - 1, 0, 0], qb[n - 1, 1, 5] = (float(x) for x in ("nan", "-inf", "inf", "nan"))
    ob, lseb = api.paged_attn(qb, *args, with_lse=True)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    for t in range(n):
        for h in range(2):
            if torch.isfinite(qb[t, h]).all() or kv - n + t < 0:     # (before the first position: sees nothing)
                assert torch.equal(ob[t, h], o[t, h]) and torch.equal(lseb[t, h], lse[t, h])
            else:
                assert torch.isnan(ob[t, h]).all() and torch.isnan(lseb[t, h])
    if kv < n:
        assert torch.isneginf(lseb[:n - kv]).all() and (ob[:n - kv] == 0).all()


def served(cu, T):
    """The sequences that a cu_q leaves in: those before the first whose entries decrease."""
    down = [b for b in range(len(cu) - 1) if cu[b + 1] < cu[b]]
    return [b for b in range(down[0]) if 0 <= cu[b] and cu[b + 1] <= T]


def random_cu(g, B, T):
    cu = torch.randint(0, T + 1, (B + 1,), generator=g).sort().values
    for i in torch.randint(0, B + 1, (max(1, B // 20),), generator=g).tolist():
        cu[i] = int(torch.randint(-2, T + 5, (1,), generator=g))
    return cu.tolist()


G = torch.Generator().manual_seed(77)
DOWN = [([0, 5, 3], 5), ([5, 3, 4], 5), ([0, 2, 1, 9], 9), ([0, 5, 3, 3, 8], 8), ([0, 5, 3, 8, 8, 9, 12], 12), ([0, 100, 2, 9, 9], 9), ([4, 2, 2, 6], 6),
        ([0, 300, 0, 300, 0, 300, 300], 300), ([0, 150] * 40 + [150, 170], 170), ([0, 1] * 250 + [1, 2], 2),
        (list(range(600)) + [100, 900], 900), (list(range(0, 500, 2)) + [499, 499, 498, 500], 500),
        (random_cu(G, 50, 200), 200), (random_cu(G, 700, 900), 900), (random_cu(G, 33, 40), 40)]


@pytest.mark.parametrize("cu,T", DOWN)
@pytest.mark.parametrize("window", [0, 20])
def test_sequences_behind_a_decreasing_entry_are_left_out(cu, T, window):
    # they could claim rows of earlier ones
    B, page, H, Hkv, d = len(cu) - 1, 16, 2, 1, 64
    g = torch.Generator().manual_seed(B)
    kv = torch.randint(0, 50, (B,), generator=g).tolist()
    table = torch.randperm(4 * B, generator=g).view(B, 4)
    kc, vc = (torch.randn(4 * B, page, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, H, d, generator=g).to(torch.bfloat16)
    out = torch.full((T, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
    args = (kc.cuda(), vc.cuda(), table.to(torch.int32).cuda(), ints(*cu), ints(*kv))
    o, _ = api.paged_attn(q.cuda(), *args, window=window, sinks=3, out=out)
    torch.cuda.synchronize()
    assert api.gca_get_status() == BAD_INDEX
    left = torch.ones(T, dtype=torch.bool)
    for b in served(cu, T):
        n, rows = cu[b + 1] - cu[b], slice(cu[b], cu[b + 1])
        left[rows] = False
        k, v = (x[table[b]].flatten(0, 1)[:kv[b]] for x in (kc, vc))
        pos = torch.arange(kv[b] - n, kv[b])
        blind = min(n, max(0, n - kv[b]))            # tokens before the first position see nothing
        assert (o[rows][:blind] == 0).all()
        if blind < n:
            ro, _, bo, _ = ref.rows(q[rows][blind:], k, v, pos[blind:], torch.arange(kv[b]), window, 3)
            ref.within("o of sequence %d" % b, o[rows][blind:], ro, bo)
    assert (o[left.cuda()] == 3.0).all()
    # the append: a row of the cache is as it was, or one of those that its sequence claims for this place
    claims = {}
    for b in range(B):
        if 0 <= cu[b] <= cu[b + 1] <= T:
            for i in range(cu[b], cu[b + 1]):
                p = kv[b] - cu[b + 1] + i
                claims.setdefault(i, []).append((int(table[b, p // page]), p % page) if p >= 0 else None)
    kn = torch.randn(T, Hkv, d, generator=g).to(torch.bfloat16)
    api.paged_append(kn.cuda(), kn.cuda(), *args)
    torch.cuda.synchronize()
    assert api.gca_get_status() == BAD_INDEX
    got, want = args[0].cpu(), kc.clone()
    for i, places in claims.items():
        hit = [x for x in places if x and torch.equal(got[x], kn[i])]
        assert len(hit) == 1 or (not hit and None in places)
        for x in hit:
            want[x] = kn[i]
    assert torch.equal(got, want)


def test_gradients_need_the_forwards_lse():
    q, k, v, g = (torch.ones(1, 8, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    o, lse = api.swa_sink_fwd(q, k, v, window=4, sinks=0, with_lse=False)
    with pytest.raises(ValueError, match="lse"):
        api.swa_sink_bwd(q, k, v, o, lse, g, window=4, sinks=0)
