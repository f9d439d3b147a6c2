"""The 64-bit reference of the transformed scores, against differences and simple cases, and what
the entries refuse (no GPU needed)."""
import ctypes
import math

import pytest
import torch

from retrieval_sparse_attention_gb300 import _lib, api

import score_reference as ref

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from retrieval_sparse_attention_gb300 import build
    build.build()
    return _lib.load()


def small(seed, B=1, L=9, H=4, Hkv=2, d=3):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, L, h, d, generator=g, dtype=torch.float64) for h in (H, Hkv, Hkv, H)]


@pytest.mark.parametrize("cap,slopes", [(1.5, None), (0.0, [0.5, 0.1, -0.2, 2.0])])
def test_gradients_are_the_differences_of_the_forward(cap, slopes):
    q, k, v, g = small(1)
    slopes = None if slopes is None else torch.tensor(slopes)
    f = lambda *x: (ref.forward(*x, 4, 1, cap, slopes)[0] * g).sum()  # noqa: E731
    o, lse, _, _ = ref.forward(q, k, v, 4, 1, cap, slopes)
    grads, _ = ref.backward(q, k, v, o, lse, g, 4, 1, cap, slopes)
    for i, x in enumerate((q, k, v)):
        for at in [(0, 0, 0, 0), (0, 3, 1, 2), (0, 8, 0, 1), (0, 5, 1, 0)]:
            old, h = x[at].item(), 1e-5
            x[at] = old + h
            up = f(q, k, v)
            x[at] = old - h
            down = f(q, k, v)
            x[at] = old
            # central differences: h^2 of the third derivative, a few 1e-9 here, and rounding 1e-16 / h
            assert abs((up - down).item() / (2 * h) - grads[i][at].item()) < 1e-7


def test_a_hand_worked_pair():
    # two tokens, one dimension: token 1 sees scores 2 tanh(3/2) and 2 tanh(-1/2), or 3 - 0.25 and -1
    q = torch.tensor([1.0, 1.0]).view(1, 2, 1, 1)
    k = torch.tensor([3.0, -1.0]).view(1, 2, 1, 1)
    v = torch.tensor([1.0, 0.0]).view(1, 2, 1, 1)
    o = ref.forward(q, k, v, 5, 0, 2.0)[0][0, 1, 0, 0]
    assert abs(o - 1 / (1 + math.exp(2 * math.tanh(-0.5) - 2 * math.tanh(1.5)))) < 1e-14
    o = ref.forward(q, k, v, 5, 0, 0.0, torch.tensor([0.25]))[0][0, 1, 0, 0]
    assert abs(o - 1 / (1 + math.exp(-1 - 2.75))) < 1e-14


@pytest.mark.parametrize("softcap,slopes,want", [
    (-1.0, None, INVALID), (float("nan"), None, INVALID), (float("inf"), None, INVALID),
    (0.0, 0x10004, INVALID), (2.0 ** -11, None, UNSUPPORTED), (1025.0, None, UNSUPPORTED),
    (5.0, 0x10000, UNSUPPORTED), (5.0, None, WORKSPACE), (0.0, 0x10000, WORKSPACE), (0.0, None, WORKSPACE)])
def test_refusals(lib, softcap, slopes, want):
    s = _lib.GcaScore(softcap, slopes)
    p = api.make_swa_sink_params(B=1, L=5000, H=2, d=64, window=64)
    assert lib.gca_swa_sink_fwd_scored(ctypes.byref(p), ctypes.byref(s), *[FAKE] * 5, None, 0, None) == want
    assert lib.gca_swa_sink_bwd_scored(ctypes.byref(p), ctypes.byref(s), *[FAKE] * 9, None, 0, None) == want
    p = api.make_paged_params(B=1, total_q=1, Hkv=2, d=64, page=16, n_pages=4, table_width=2)
    assert lib.gca_paged_attn_scored(ctypes.byref(p), ctypes.byref(s), *[FAKE] * 7, None, None, 0, None) == want


def test_no_struct_is_the_plain_call(lib):
    p = api.make_swa_sink_params(B=1, L=5000, H=2, d=64, window=64)
    assert lib.gca_swa_sink_fwd_scored(ctypes.byref(p), None, *[FAKE] * 5, None, 0, None) == WORKSPACE
    assert lib.gca_swa_sink_fwd_scored(None, None, *[FAKE] * 5, None, 0, None) == INVALID


def test_slopes_of_the_binding():
    with pytest.raises(ValueError, match="slopes"):
        api._score(0.0, torch.zeros(3), 4, -1)
    with pytest.raises(TypeError, match="slopes"):
        api._score(0.0, torch.zeros(4, dtype=torch.float64), 4, -1)
    with pytest.raises(ValueError, match="slopes"):
        api._score(0.0, torch.zeros(8)[::2], 4, -1)
    with pytest.raises(ValueError, match="device"):
        api._score(0.0, torch.zeros(4), 4, 0)            # (a CPU tensor next to CUDA ones)
    assert api._score(0.0, None, 4, 0) is None
    assert api._score(torch.tensor(2.5), None, 4, 0).softcap == 2.5
