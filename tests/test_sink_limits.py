"""The sizes that the windowed attention with sinks takes (no GPU needed): its kernels count
their steps in 32 bits, so every stream of a call that is not refused has to fit."""
import ctypes
import random

import pytest

from retrieval_sparse_attention_gb300 import _lib, api

UNSUPPORTED, WORKSPACE = 2, 3
FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    from retrieval_sparse_attention_gb300 import build
    build.build()
    return _lib.load()


def streams(B, L, H, Hkv, d, window, sinks):
    """Steps of the query-major gradients: 64-key tiles of each (row, key head, query tile)."""
    W = min(window, L)
    ns = min(sinks, L) if W < L else 0
    TM = min(128 * Hkv // H, L)
    total = 0
    for p0 in range(0, L, TM):
        p1 = min(L, p0 + TM) - 1
        k0 = max(0, p0 - W + 1) >> 6
        total += min((ns + 63) >> 6, k0) + (p1 >> 6) - k0 + 1
    return B * Hkv * total


# groups that do not divide 128 (one token a query tile): twice the key-major steps
@pytest.mark.parametrize("B,L,H,Hkv,window", [(1, 1000000, 65, 1, 150000), (8, 131072, 272, 4, 40000)])
def test_gradients_whose_query_major_steps_pass_32_bits_are_refused(lib, B, L, H, Hkv, window):
    assert streams(B, L, H, Hkv, 64, window, 0) >= 2 ** 31
    p = api.make_swa_sink_params(B=B, L=L, H=H, Hkv=Hkv, d=64, window=window)
    assert api.gca_swa_sink_bwd_workspace_size(p) == 0
    assert lib.gca_swa_sink_bwd(ctypes.byref(p), *[FAKE] * 9, None, 0, None) == UNSUPPORTED


def test_steps_of_supported_gradients_fit_32_bits():
    rng = random.Random(3)
    refused = 0
    for _ in range(60):
        Hkv = rng.choice([1, 2, 3])
        H = Hkv * rng.choice([43, 50, 65, 70, 100, 128])
        L = rng.randrange(30000, 200000)
        B = max(1, int(2 ** rng.uniform(0, 9)))
        while B * L * H >= 2 ** 31:
            B = max(1, B // 2)
            L = L * 3 // 4
        window, sinks = rng.randrange(1, 2 * L), rng.choice([0, 4, 1000, L])
        p = api.make_swa_sink_params(B=B, L=L, H=H, Hkv=Hkv, d=64, window=window, sinks=sinks)
        if api.gca_swa_sink_bwd_workspace_size(p) == 0:
            refused += 1
        else:
            n = streams(B, L, H, Hkv, 64, window, sinks)
            assert n + n // 152 + 200 < 2 ** 31, (B, L, H, Hkv, window, sinks)      # a share past the end
    assert 0 < refused < 60


def key_major_steps(B, L, H, window, sinks):
    """64-query blocks of each (row, query head, 128-key tile)."""
    W = min(window, L)
    ns = min(sinks, L) if W < L else 0
    last = (L - 1) >> 6
    return B * H * sum((last if s0 < ns else min(L - 1, s0 + 127 + W - 1) >> 6) - s0 // 64 + 1 for s0 in range(0, L, 128))


def forward_tiles(B, L, H, Hkv, window, sinks):
    W = min(window, L)
    ns = min(sinks, L) if W < L else 0
    TM = min(128 * Hkv // H, L)
    total = 0
    for p0 in range(0, L, TM):
        k0 = max(0, p0 - W + 1) >> 7
        total += min((ns + 127) >> 7, k0) + ((min(L, p0 + TM) - 1) >> 7) - k0 + 1
    return B * Hkv * total


def test_the_forward_has_limits_of_its_own(lib):
    # full causal attention over 1M tokens: 0.54e9 key tiles and 1.07e9 gradient steps, and its double
    for H, Hkv, bwd in ((16, 4, True), (32, 8, False)):
        p = api.make_swa_sink_params(B=1, L=2 ** 20, H=H, Hkv=Hkv, d=128, window=2 ** 20)
        assert api.gca_swa_sink_fwd_workspace_size(p) > 0
        assert (api.gca_swa_sink_bwd_workspace_size(p) > 0) == bwd
        # (a workspace that is missing is what stops the call)
        assert lib.gca_swa_sink_fwd(ctypes.byref(p), *[FAKE] * 5, None, 0, None) == WORKSPACE
        got = lib.gca_swa_sink_bwd(ctypes.byref(p), *[FAKE] * 9, None, 0, None)
        assert got == (WORKSPACE if bwd else UNSUPPORTED)


def test_limits_follow_the_counts():
    # what is taken fits 32 bits with a share past the end; what is refused is not far below
    rng = random.Random(4)
    seen = set()
    for _ in range(150):
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 3, 7, 12, 16, 48, 70, 128])
        L = rng.randrange(20000, 400000)
        B = int(2 ** rng.uniform(0, 10))
        while B * L * H >= 2 ** 31 and B > 1:
            B //= 2
        if B * L * H >= 2 ** 31:
            continue
        window, sinks = rng.choice([rng.randrange(1, L), L, 3000]), rng.choice([0, 4, 500, L // 2, L])
        p = api.make_swa_sink_params(B=B, L=L, H=H, Hkv=Hkv, d=64, window=window, sinks=sinks)
        fwd = forward_tiles(B, L, H, Hkv, window, sinks)
        bwd = max(key_major_steps(B, L, H, window, sinks), streams(B, L, H, Hkv, 64, window, sinks))
        for n, size in ((fwd, api.gca_swa_sink_fwd_workspace_size(p)), (bwd, api.gca_swa_sink_bwd_workspace_size(p))):
            if size:
                assert n + n // 152 + 400 < 2 ** 31, (B, L, H, Hkv, window, sinks)
            else:
                assert n > 1.8e9, (B, L, H, Hkv, window, sinks)
            seen.add((n == fwd, size > 0))
    assert len(seen) == 4


def paged(**kw):
    base = dict(B=4, total_q=0, max_q=0, H=0, Hkv=2, d=64, page=16, n_pages=10, table_width=3, window=0, sinks=0,
                dtype=0, attn_scale=0.0, q_stride=0, kv_stride=0)
    base.update(kw)
    return _lib.GcaPagedParams(**base)


def test_the_append_needs_no_query_heads(lib):
    p = paged()
    # nothing to write: only the parameters are checked
    assert lib.gca_paged_append(ctypes.byref(p), *[None] * 7, None) == 0
    assert lib.gca_paged_attn(ctypes.byref(p), *[None] * 9, 0, None) == 1


def test_the_append_has_no_limit_of_tiles(lib):
    # 2^30 new tokens over 2^29 cached ones are too many key tiles to attend over, not too many rows
    p = paged(B=3, total_q=2 ** 30, H=2, Hkv=2, n_pages=2 ** 27, table_width=2 ** 25)
    assert lib.gca_paged_attn(ctypes.byref(p), *[None] * 9, 0, None) == UNSUPPORTED
    # (tensors that are missing are what stops the call)
    assert lib.gca_paged_append(ctypes.byref(p), *[None] * 7, None) == 1
    assert lib.gca_paged_append(ctypes.byref(paged(page=24)), *[None] * 7, None) == UNSUPPORTED
    assert lib.gca_paged_append(ctypes.byref(paged(Hkv=0)), *[None] * 7, None) == 1


def test_positions_of_new_tokens_fit_32_bits(lib):
    # the first of n tokens stands at -n where nothing is cached, and its window 2^30 before that
    for n, max_q, code in ((2 ** 30 + 1, 0, UNSUPPORTED), (2 ** 30, 0, 1), (2 ** 31 - 1, 1000, 1)):
        assert -min(n, max_q or n) - 2 ** 30 >= -2 ** 31 or code == UNSUPPORTED
        p = paged(B=1, total_q=n, max_q=max_q, H=1, Hkv=1)
        # (tensors that are missing are what stops the others)
        assert lib.gca_paged_attn(ctypes.byref(p), *[None] * 9, 0, None) == code
