"""The 64-bit reference of the windowed attention with sinks against central
differences and against autograd, and the C ABI's refusals (no GPU needed)."""
import ctypes

import pytest
import torch

from retrieval_sparse_attention_gb300 import _lib, api
from retrieval_sparse_attention_gb300._lib import GcaPagedParams, GcaSwaSinkParams

import sink_reference as ref

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from retrieval_sparse_attention_gb300 import build
    build.build()
    return _lib.load()


@pytest.mark.parametrize("window,sinks,H,Hkv", [(3, 2, 2, 1), (1, 0, 2, 2), (4, 1, 3, 1), (50, 4, 2, 1)])
def test_reference_gradients(window, sinks, H, Hkv):
    g = torch.Generator().manual_seed(window)
    L, d = 9, 4
    q, k, v = (torch.randn(1, L, h, d, generator=g, dtype=torch.float64) for h in (H, Hkv, Hkv))
    dout = torch.randn(1, L, H, d, generator=g, dtype=torch.float64)
    o, lse, _, _ = ref.forward(q, k, v, window, sinks)
    grads, _ = ref.backward(q, k, v, o, lse, dout, window, sinks)

    def loss(q, k, v):
        return float((ref.forward(q, k, v, window, sinks)[0] * dout).sum())
    h = 1e-5
    for x, gx in zip((q, k, v), grads):
        flat, num = x.view(-1), torch.empty_like(x).view(-1)
        for i in range(flat.numel()):
            old = float(flat[i])
            flat[i] = old + h
            up = loss(q, k, v)
            flat[i] = old - h
            num[i] = (up - loss(q, k, v)) / (2 * h)
            flat[i] = old
        assert (num - gx.reshape(-1)).abs().max() < 1e-8 * 10
    xs = [x.clone().requires_grad_() for x in (q, k, v)]
    (ref.forward(*xs, window, sinks)[0] * dout).sum().backward()
    for x, gx in zip(xs, grads):
        assert (x.grad - gx).abs().max() < 1e-12


def test_reference_rows_without_a_visible_key():
    x = torch.randn(3, 1, 4, dtype=torch.float64)
    o, lse, _, _ = ref.rows(x, x[:1], x[:1], torch.arange(-2, 1), torch.arange(1), 0, 0)
    assert (o[:2] == 0).all() and torch.isneginf(lse[:2]).all() and torch.isfinite(lse[2]).all()


def sink(**kw):
    base = dict(B=2, L=300, H=4, Hkv=2, d=64, window=128, sinks=4, dtype=0, attn_scale=0.0,
                q_stride=0, kv_stride=0)
    base.update(kw)
    return GcaSwaSinkParams(**base)


def call_fwd(lib, p, q=FAKE, ws=FAKE, n=1 << 40):
    return lib.gca_swa_sink_fwd(ctypes.byref(p) if p is not None else None, q, FAKE, FAKE, FAKE, None, ws, n, None)


BAD_SINK = [(dict(B=0), INVALID), (dict(L=0), INVALID), (dict(window=0), INVALID), (dict(sinks=-1), INVALID),
            (dict(H=3), INVALID), (dict(Hkv=0), INVALID), (dict(dtype=5), INVALID), (dict(attn_scale=-1.0), INVALID),
            (dict(attn_scale=float("nan")), INVALID), (dict(attn_scale=float("inf")), INVALID),
            (dict(q_stride=255), INVALID), (dict(q_stride=8), INVALID), (dict(kv_stride=-128), INVALID),
            (dict(kv_stride=132), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
            (dict(d=256), UNSUPPORTED), (dict(H=258, Hkv=2), UNSUPPORTED), (dict(B=1 << 20, L=1 << 20), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_SINK)
def test_sink_refusals(lib, kw, code):
    p = sink(**kw)
    assert call_fwd(lib, p) == code
    assert lib.gca_swa_sink_bwd(ctypes.byref(p), *[FAKE] * 10, 1 << 40, None) == code
    assert lib.gca_swa_sink_fwd_workspace_size(ctypes.byref(p)) == 0
    assert lib.gca_swa_sink_bwd_workspace_size(ctypes.byref(p)) == 0


def test_sink_pointers_and_workspaces(lib):
    p = sink()
    assert call_fwd(lib, None) == INVALID
    assert call_fwd(lib, p, q=None) == INVALID
    assert call_fwd(lib, p, q=ctypes.c_void_p(0x10008)) == INVALID
    nf, nb = lib.gca_swa_sink_fwd_workspace_size(ctypes.byref(p)), lib.gca_swa_sink_bwd_workspace_size(ctypes.byref(p))
    assert nf > 0 and nb > 0 and lib.gca_swa_sink_fwd_workspace_size(None) == 0
    for ws, n in ((None, nf), (FAKE, nf - 1), (ctypes.c_void_p(0x10080), nf)):
        assert call_fwd(lib, p, ws=ws, n=n) == WORKSPACE
    for ws, n in ((None, nb), (FAKE, nb - 1), (ctypes.c_void_p(0x10080), nb)):
        assert lib.gca_swa_sink_bwd(ctypes.byref(p), *[FAKE] * 9, ws, n, None) == WORKSPACE
    for i in range(9):
        args = [FAKE] * 9
        args[i] = None
        assert lib.gca_swa_sink_bwd(ctypes.byref(p), *args, FAKE, nb, None) == INVALID


def paged(**kw):
    base = dict(B=3, total_q=10, max_q=4, H=4, Hkv=2, d=64, page=16, n_pages=9, table_width=5, window=0,
                sinks=0, dtype=0, attn_scale=0.0, q_stride=0, kv_stride=0)
    base.update(kw)
    return GcaPagedParams(**base)


BAD_PAGED = [(dict(B=0), INVALID), (dict(total_q=-1), INVALID), (dict(max_q=-1), INVALID), (dict(n_pages=0), INVALID),
             (dict(table_width=0), INVALID), (dict(page=0), INVALID), (dict(window=-1), INVALID),
             (dict(sinks=-1), INVALID), (dict(H=5), INVALID), (dict(dtype=9), INVALID), (dict(dtype=1), UNSUPPORTED),
             (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
             (dict(B=70000), UNSUPPORTED), (dict(table_width=1 << 29), UNSUPPORTED), (dict(q_stride=100), INVALID),
             (dict(kv_stride=64), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_PAGED)
def test_paged_refusals(lib, kw, code):
    p = paged(**kw)
    assert lib.gca_paged_append(ctypes.byref(p), *[FAKE] * 7, None) == code
    assert lib.gca_paged_attn(ctypes.byref(p), *[FAKE] * 7, None, FAKE, 1 << 40, None) == code
    assert lib.gca_paged_attn_workspace_size(ctypes.byref(p)) == 0


def test_paged_pointers_workspace_and_nothing_to_do(lib):
    p = paged()
    n = lib.gca_paged_attn_workspace_size(ctypes.byref(p))
    assert n > 0
    for i in range(7):
        args = [FAKE] * 7
        args[i] = None
        assert lib.gca_paged_append(ctypes.byref(p), *args, None) == INVALID
        assert lib.gca_paged_attn(ctypes.byref(p), *args, None, FAKE, n, None) == INVALID
    for ws, m in ((None, n), (FAKE, n - 1), (ctypes.c_void_p(0x10080), n)):
        assert lib.gca_paged_attn(ctypes.byref(p), *[FAKE] * 7, None, ws, m, None) == WORKSPACE
    assert lib.gca_paged_attn(ctypes.byref(p), *[FAKE] * 7, ctypes.c_void_p(0x10004), FAKE, n, None) == INVALID
    # no rows at all: nothing is enqueued, and no pointer is looked at
    p0 = paged(total_q=0)
    assert lib.gca_paged_append(ctypes.byref(p0), *[None] * 7, None) == OK
    assert lib.gca_paged_attn(ctypes.byref(p0), *[None] * 7, None, None, 0, None) == OK
    assert lib.gca_last_launch_count() == 0
    assert lib.gca_paged_append(None, *[FAKE] * 7, None) == INVALID
    assert lib.gca_paged_attn(None, *[FAKE] * 7, None, FAKE, n, None) == INVALID


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.swa_sink_fwd(x, x, x, window=4, sinks=1)
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.paged_attn(x[0], c, c, t, torch.tensor([0, 8], dtype=torch.int32), torch.tensor([8], dtype=torch.int32))
