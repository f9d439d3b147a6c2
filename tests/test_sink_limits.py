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
