"""What the binding of the windowed attention with sinks and of its paged cache makes of its
arguments (no GPU needed)."""
import pytest
import torch

from retrieval_sparse_attention_gb300 import api


@pytest.fixture(scope="module", autouse=True)
def lib():
    from retrieval_sparse_attention_gb300 import build
    build.build()


def dense(window, sinks=0, attn_scale=0.0, L=40):
    x = torch.zeros(1, L, 2, 64, dtype=torch.bfloat16)
    return api._swa_sink_args(x, x, x, window, sinks, attn_scale)[0]


def paged(window=0, sinks=0, attn_scale=0.0, max_q=0):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    c = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    return api._paged_args(q, c, c, i(3, 2), i(4), i(3), True, max_q, window, sinks, attn_scale)[0]


def test_a_tensor_that_changes_is_read_anew():
    w, s, a = torch.tensor(30), torch.tensor(4), torch.tensor(0.5)
    for f in (dense, paged):
        w.fill_(30), s.fill_(4), a.fill_(0.5)
        p = f(w, s, a)
        assert (p.window, p.sinks, p.attn_scale) == (30, 4, 0.5)
        w.fill_(20), s.fill_(3), a.fill_(0.25)
        p = f(w, s, a)
        assert (p.window, p.sinks, p.attn_scale) == (20, 3, 0.25)
    m = torch.tensor(2)
    assert paged(max_q=m).max_q == 2
    m.fill_(3)
    assert paged(max_q=m).max_q == 3


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 64 + 7])
def test_numbers_beyond_32_bits_mean_all_tokens(big):
    for f in (dense, paged):
        p = f(big, big)
        assert p.window >= 40 and p.sinks >= 40
    assert paged(max_q=big).max_q >= 5


def test_no_number_is_cut_to_32_bits():
    for kw in (dict(window=2 ** 32 + 5), dict(window=torch.tensor(2 ** 32 + 5)), dict(L=2 ** 32 + 8), dict(q_stride=2 ** 32 + 128), dict(sinks=-2 ** 32)):
        with pytest.raises(ValueError):
            api.make_swa_sink_params(**{**dict(B=1, L=8, H=2, d=64, window=4), **kw})
    base = dict(B=1, total_q=1, Hkv=2, d=64, page=16, n_pages=4, table_width=2)
    for kw in (dict(window=-2 ** 32 + 1), dict(total_q=2 ** 32 + 1), dict(n_pages=2 ** 31)):
        with pytest.raises(ValueError):
            api.make_paged_params(**{**base, **kw})
    with pytest.raises(ValueError):
        dense(-2 ** 32 + 9)


def test_floats_are_no_counts():
    dense(30)                       # (a kept plan for 30 does not answer for 30.0)
    paged(30)
    for f in (dense, paged):
        with pytest.raises(TypeError):
            f(30.0)
        with pytest.raises(TypeError):
            f(30, 4.0)
    assert dense(True).window == 1


def test_a_missing_lse_is_named():
    # (as from a forward without it)
    with pytest.raises(ValueError, match="lse"):
        api._dense(None, (1, 8, 2), torch.float32, "lse")
