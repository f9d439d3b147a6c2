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
