"""Rotary positions and pages without a GPU: the list model that the GPU tests compare with, the
rotary tables, and what the entries refuse."""
import ctypes
import math
import random

import pytest
import torch

from retrieval_sparse_attention_gb300 import _lib, api

from page_model import Pages

INVALID, UNSUPPORTED = 1, 2
FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    from retrieval_sparse_attention_gb300 import build
    build.build()
    return _lib.load()


def counted(m):
    refs = [0] * m.n
    for row in m.table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    return refs


def test_the_model_keeps_its_counts():
    r = random.Random(1)
    for _ in range(20):
        m = Pages(5, 8, 24, 16)
        for _ in range(30):
            kind = r.randrange(4)
            if kind < 2:
                cu = [0]
                for _ in range(5):
                    cu.append(cu[-1] + r.choice([0, 1, 1, 7, 40]))
                m.reserve(cu, r.choice([0, 20, 40]), r.choice([0, 3, 17]))
            elif kind == 2:
                m.fork([r.randrange(-1, 5) for _ in range(5)])
            else:
                m.compact(r.choice([1, 3, 24]))
            assert counted(m) == m.refs
            for b in range(5):                          # an unfinished page is held once
                n = -1 - m.kv[b] if m.kv[b] < 0 else m.kv[b]
                if n % 16 and m.table[b][n // 16] >= 0:
                    assert m.refs[m.table[b][n // 16]] == 1


def test_a_worked_reservation():
    m = Pages(2, 4, 4, 16)
    m.reserve([0, 20, 21])
    assert m.table == [[0, 1, -1, -1], [2, -1, -1, -1]] and m.kv == [20, 1]
    m.reserve([0, 30, 46])                              # two pages and one, of one that is left
    assert m.kv == [-21, -2] and m.status == 7 and m.table[0] == [0, 1, -1, -1]
    m.fork([-1, 1])                                     # the first ends
    m.reserve([0, 0, 16])
    assert m.table[1] == [2, 0, -1, -1] and m.kv == [0, 17]


def test_rope_tables():
    f = api.rope_freqs(64, device="cpu")
    assert f.dtype == torch.int64 and f.shape == (32,)
    inv = 10000.0 ** -(torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    got = f.double() / 2.0 ** 64 * 2 * math.pi
    assert (got - inv).abs().max() <= 2.0 ** -51        # a rounding of 2 pi, one of the quotient
    # whole turns do not show, half a turn is one number
    t = api.rope_table([2 * math.pi, math.pi, -math.pi, 0.0], device="cpu")
    assert t.tolist() == [0, -2 ** 63, -2 ** 63, 0] or t.tolist()[1] in (-2 ** 63, 2 ** 63 - 1)
    assert torch.equal(api.rope_freqs(64, scaling="linear", factor=4.0, device="cpu"), api.rope_table(inv / 4, "cpu"))
    n = api.rope_freqs(64, scaling="ntk", factor=4.0, device="cpu").double() / f.double()
    assert abs(n[0] - 1) < 1e-12 and abs(n[31] - 0.25) < 1e-9
    y = api.rope_freqs(64, scaling="yarn", factor=4.0, trained_len=4096, device="cpu").double() / f.double()
    turns = 4096 * inv / (2 * math.pi)
    assert (y[turns >= 32] - 1).abs().max() < 1e-9 and (y[turns <= 1] - 0.25).abs().max() < 1e-9
    assert (y[1:] <= y[:-1] + 1e-9).all()
    for kw in (dict(scaling="other"), dict(factor=0.0), dict(base=1.0), dict(scaling="yarn"),
               dict(scaling="yarn", trained_len=100, beta_fast=1.0)):
        with pytest.raises(ValueError):
            api.rope_freqs(64, device="cpu", **kw)
    for rot in (2, 5):
        with pytest.raises(ValueError):
            api.rope_freqs(rot, device="cpu")
    with pytest.raises(ValueError):
        api.rope_table([float("nan")], "cpu")


def rope_params(**kw):
    base = dict(T=4, L=4, start=0, H=2, Hkv=1, d=64, rot=64, interleaved=0, inverse=0, dtype=0, mscale=0.0, q_stride=0,
                k_stride=0, q_out_stride=0, k_out_stride=0)
    return _lib.GcaRopeParams(**{**base, **kw})


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(L=0), INVALID), (dict(start=-1), INVALID), (dict(start=2 ** 31 - 4), INVALID),
    (dict(H=0, Hkv=0), INVALID), (dict(H=-1), INVALID), (dict(dtype=2), INVALID), (dict(rot=0), INVALID),
    (dict(rot=80), INVALID), (dict(mscale=-1.0), INVALID), (dict(mscale=float("inf")), INVALID),
    (dict(q_stride=64), INVALID), (dict(k_stride=68), INVALID), (dict(q_out_stride=-8), INVALID),
    (dict(d=96, rot=96), UNSUPPORTED), (dict(rot=40), UNSUPPORTED), (dict(H=5000), UNSUPPORTED),
    (dict(q_stride=1 << 25), UNSUPPORTED), (dict(T=2 ** 31 - 1, L=1, H=4096), UNSUPPORTED), (dict(T=0), 0)])
def test_rope_refusals(lib, kw, want):
    # (a null k_out, which no call gets as far as)
    got = lib.gca_rope(ctypes.byref(rope_params(**kw)), FAKE, FAKE, FAKE, None, FAKE, None, None)
    assert got == want


def test_rope_pointers(lib):
    call = lambda p, *a: lib.gca_rope(ctypes.byref(p) if p else None, *a, None)  # noqa: E731
    assert call(None, *[FAKE] * 6) == INVALID
    for i in (0, 1, 2, 4, 5):
        for bad in (None, ODD):
            a = [FAKE, FAKE, FAKE, None, FAKE, FAKE]
            a[i] = bad
            assert call(rope_params(), *a) == INVALID
    assert call(rope_params(), FAKE, FAKE, FAKE, ODD, FAKE, FAKE) == INVALID


def test_paged_rope_append_refusals(lib):
    base = dict(B=1, total_q=4, Hkv=2, d=64, page=16, n_pages=4, table_width=2)

    def call(rope, paged=None, ptr=FAKE):
        return lib.gca_paged_rope_append(ctypes.byref(api.make_paged_params(**{**base, **(paged or {})})),
                                         ctypes.byref(rope) if rope else None, ptr, *[FAKE] * 9, None)
    assert call(None) == INVALID
    assert call(rope_params(), ptr=None) == INVALID
    assert call(rope_params(rot=72)) == INVALID
    assert call(rope_params(rot=24)) == UNSUPPORTED
    assert call(rope_params(inverse=1)) == UNSUPPORTED
    assert call(rope_params(), dict(H=0)) == INVALID
    assert call(rope_params(), dict(page=48)) == UNSUPPORTED
    assert call(rope_params(), dict(total_q=0)) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INVALID), (dict(n_pages=0), INVALID), (dict(table_width=0), INVALID), (dict(page=0), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(page=48), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(n_pages=2 ** 24 + 1), UNSUPPORTED), (dict(table_width=2 ** 26, page=16), UNSUPPORTED),
    (dict(B=4096, table_width=2 ** 20, page=16), UNSUPPORTED)])
def test_page_refusals(lib, kw, want):
    p = _lib.GcaPagesParams(**{**dict(B=2, page=16, n_pages=8, table_width=4, window=0, sinks=0), **kw})
    r = ctypes.byref(p)
    assert lib.gca_paged_reserve(r, *[FAKE] * 4, None) == want
    assert lib.gca_paged_fork(r, *[FAKE] * 5, None) == want
    assert lib.gca_paged_compact(r, 4, *[FAKE] * 3, None) == want


def test_page_pointers(lib):
    p = _lib.GcaPagesParams(B=2, page=16, n_pages=8, table_width=4, window=0, sinks=0)
    r = ctypes.byref(p)
    for bad in (None, ODD):
        for i in range(4):
            a = [FAKE] * 4
            a[i] = bad
            assert lib.gca_paged_reserve(r, *a, None) == INVALID
        for i in range(5):
            a = [FAKE] * 5
            a[i] = bad
            assert lib.gca_paged_fork(r, *a, None) == INVALID
        for i in range(3):
            a = [FAKE] * 3
            a[i] = bad
            assert lib.gca_paged_compact(r, 4, *a, None) == INVALID
            assert lib.gca_paged_copy(4096, 8, a[0], 2, a[1], a[2], None) == INVALID
        assert lib.gca_page_pool_init(8, bad, None) == INVALID
    assert lib.gca_paged_compact(r, 0, *[FAKE] * 3, None) == INVALID
    assert lib.gca_paged_compact(r, 2 ** 24 + 1, *[FAKE] * 3, None) == UNSUPPORTED
    assert lib.gca_paged_reserve(None, *[FAKE] * 4, None) == INVALID
    for bytes_, n_pages, n, want in ((0, 8, 2, INVALID), (24, 8, 2, INVALID), (4096, 0, 2, INVALID), (4096, 8, -1, INVALID),
                                     (2 ** 31, 8, 2, UNSUPPORTED), (2 ** 30, 8, 2 ** 20, UNSUPPORTED), (4096, 8, 0, 0)):
        assert lib.gca_paged_copy(bytes_, n_pages, FAKE, n, FAKE, FAKE, None) == want
    assert lib.gca_page_pool_init(0, FAKE, None) == INVALID
    assert lib.gca_page_pool_init(2 ** 24 + 1, FAKE, None) == UNSUPPORTED
    assert lib.gca_page_pool_ints(0) == 0 and lib.gca_page_pool_ints(2 ** 24 + 1) == 0
    assert lib.gca_page_pool_ints(33) == 68


def test_what_the_binding_refuses():
    q = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16)
    plan = lambda *a, **k: api._rope_plan.__wrapped__(*a, **k)  # noqa: E731
    rest = dict(pairs=32, pos=None, start=0, interleaved=False, mscale=1.0, inverse=False, inplace=False)
    p = plan(q.shape, q.stride(), None, None, q.dtype, None, **rest)
    assert (p.T, p.L, p.H, p.Hkv, p.d, p.rot) == (16, 8, 4, 0, 64, 64)
    with pytest.raises(ValueError):
        plan(q.shape, q.stride(), (2, 9, 4, 64), (2304, 256, 64, 1), q.dtype, q.dtype, **rest)
    with pytest.raises(TypeError):
        plan(q.shape, q.stride(), q.shape, q.stride(), q.dtype, torch.float32, **rest)
    with pytest.raises(ValueError):
        plan(q.shape, q.stride(), None, None, q.dtype, None, **{**rest, "pos": (16,)})
    with pytest.raises(ValueError):
        plan(q.shape, q.stride(), None, None, q.dtype, None, **{**rest, "start": 2 ** 31})
    with pytest.raises(ValueError):
        api.rope(None, None, torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError):                    # no CUDA tensors
        api.rope(q, None, torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError):
        api._rope_freqs(torch.zeros(32))
    with pytest.raises(ValueError):
        api._pages_plan((2, 4), (2,), 67, 16, 0, 0)    # no pool has so many words
    with pytest.raises(ValueError):
        api._pages_plan((2, 4), (3,), 68, 16, 0, 0)
    assert api._pages_plan((2, 4), (2,), 68, 16, 2 ** 40, 0).n_pages == 33
    with pytest.raises(ValueError):
        api.page_pool(0)
