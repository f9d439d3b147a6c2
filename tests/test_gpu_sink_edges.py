"""Calls of the windowed attention with sinks and of its paged cache that stand at the edge of
what their documentation allows."""
import pytest
import torch

from retrieval_sparse_attention_gb300 import api

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
