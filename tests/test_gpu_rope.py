"""Rotary positions on the GPU against 64 bits.

Bounds, with U = 2^-8 (bf16) or 2^-24 (fp32) for the result's rounding: the sine and cosine
are off by 2^-21.1 (bf16: the hardware's 2^-21.2 within half a turn, and an argument
off by 2^-24 of pi) or 2^-22 (fp32: two units in the last place and the argument's 2^-24),
each product and sum rounds by 2^-24: m (|x| + |y|) (2^-20.5 or 2^-21) in all."""
import math

import pytest
import torch

from retrieval_sparse_attention_gb300 import api
from retrieval_sparse_attention_gb300._lib import GcaError

pytestmark = pytest.mark.gpu


def angles(freqs, pos):
    """pos [...] x pairs -> radians, from the table in exact 64-bit arithmetic."""
    return (pos.long()[..., None] * freqs).double() * (2 * math.pi / 2.0 ** 64)      # (int64 products wrap)


def reference(x, freqs, pos, inter, m=1.0, sign=1):
    x = x.double().cpu()
    a = sign * angles(freqs.cpu(), pos.cpu())[..., None, :]
    rot = 2 * freqs.numel()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    u, w = x[..., first], x[..., second]
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = m * (u * a.cos() - w * a.sin()), m * (u * a.sin() + w * a.cos())
    mag[..., first] = mag[..., second] = m * (u.abs() + w.abs())
    return y, mag


def check(got, x, freqs, pos, inter, m=1.0, sign=1):
    want, mag = reference(x, freqs, pos, inter, m, sign)
    unit, trig = (2.0 ** -8, 2.0 ** -20.5) if x.dtype == torch.bfloat16 else (2.0 ** -24, 2.0 ** -21)
    assert got.dtype == x.dtype and got.shape == x.shape
    err = (got.double().cpu() - want).abs() - (unit * want.abs() + (1 + unit) * trig * mag)
    assert float(err.max()) <= 0, float(err.max())


def normal(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


# B, L, H, Hkv, d, rot: one token, more slots than a warp takes at once, one head, all head sizes, part of a head
SHAPES = [(1, 1, 1, 1, 64, 64), (1, 517, 12, 12, 64, 64), (2, 33, 16, 4, 128, 64), (3, 7, 5, 1, 32, 16), (1, 40, 3, 2, 256, 256),
          (1, 9, 40, 3, 128, 128), (2, 5, 1, 1, 256, 16), (1, 300, 7, 0, 64, 48), (1, 64, 0, 2, 128, 112)]


@pytest.mark.parametrize("B,L,H,Hkv,d,rot", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_element(B, L, H, Hkv, d, rot, inter, dtype):
    q = normal(B, L, H, d, seed=1, dtype=dtype) if H else None
    k = normal(B, L, Hkv, d, seed=2, dtype=dtype) if Hkv else None
    freqs = api.rope_freqs(rot)
    pos = 1000 + torch.arange(L).expand(B, L)
    for f, sign in ((api.rope, 1), (api.rope_bwd, -1)):
        a, b = f(q, k, freqs, start=1000, interleaved=inter, mscale=1.25)
        for x, y in ((q, a), (k, b)):
            assert (x is None) == (y is None)
            if x is not None:
                check(y, x, freqs, pos, inter, 1.25, sign)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_positions_far_and_negative(dtype):
    pos = torch.tensor([0, 1, -1, 7, 2 ** 20, 10 ** 9, 2 ** 31 - 1, -2 ** 31, 123456789, 5, 5, -4000], dtype=torch.int32)
    q, k = normal(12, 4, 64, dtype=dtype), normal(12, 2, 64, seed=3, dtype=dtype)
    for scaling in (dict(), dict(scaling="yarn", factor=8.0, trained_len=4096), dict(scaling="ntk", factor=2.0)):
        freqs = api.rope_freqs(64, **scaling)
        a, b = api.rope(q, k, freqs, positions=pos.cuda())
        check(a, q, freqs, pos, False)
        check(b, k, freqs, pos, False)
    a, b = api.rope(q.view(2, 6, 4, 64), k.view(2, 6, 2, 64), freqs, positions=pos.view(2, 6).cuda(), interleaved=True)
    check(a.view(12, 4, 64), q, freqs, pos, True)


def test_quarter_turns_are_exact_in_fp32():
    # angles of whole quarter turns: the sines and cosines are 0 and 1
    x = normal(9, 1, 32, seed=4, dtype=torch.float32)
    freqs = api.rope_table([math.pi / 2] * 16)
    y, _ = api.rope(x, None, freqs)
    u, w = x[..., :16], x[..., 16:]
    for t in range(9):
        want = [(u, w), (-w, u), (-u, -w), (w, -u)][t % 4]
        assert (y[t] - torch.cat([v[t] for v in want], -1)).abs().max() <= 2.0 ** -30 * 8


def test_gradient_is_the_transpose():
    # <rope(x), g> = <x, rope_bwd(g)>, and differences of a smooth function
    x, g = normal(40, 3, 64, seed=5, dtype=torch.float32), normal(40, 3, 64, seed=6, dtype=torch.float32)
    freqs = api.rope_freqs(32)
    y, _ = api.rope(x, None, freqs, start=77, mscale=0.5)
    dx, _ = api.rope_bwd(g, None, freqs, start=77, mscale=0.5)
    a, b = (y.double() * g.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(a - b) <= 2.0 ** -20 * (y.double().abs() * g.double().abs()).sum()
    for at in ((0, 0, 0), (39, 2, 16), (20, 1, 31), (5, 0, 40)):
        z = x.clone()
        z[at] += 1.0
        d, _ = api.rope(z, None, freqs, start=77, mscale=0.5)
        diff = ((d - y).double() * g.double()).sum()     # (linear: any step will do; y and d are off by 2^-21 of a few units)
        assert abs(diff - dx[at]) <= 2.0 ** -17


def test_packed_projection_and_in_place():
    B, L, H, Hkv, d = 2, 50, 4, 2, 64
    x = normal(B, L, (H + 2 * Hkv) * d, seed=7)
    q, k, v = (y.unflatten(-1, (-1, d)) for y in x.split([H * d, Hkv * d, Hkv * d], -1))
    kept = x.clone()
    freqs = api.rope_freqs(64)
    a, b = api.rope(q, k, freqs)
    assert torch.equal(x, kept) and a.is_contiguous() and b.is_contiguous()
    pos = torch.arange(L).expand(B, L)
    check(a, q, freqs, pos, False)
    c, e = api.rope(q, k, freqs, inplace=True)
    assert c is q and e is k
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(v, kept.split([H * d, Hkv * d, Hkv * d], -1)[2].unflatten(-1, (-1, d)))


def test_no_tokens_and_refusals():
    freqs = api.rope_freqs(64)
    a, b = api.rope(normal(0, 4, 64), normal(0, 2, 64), freqs)
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)
    a, _ = api.rope(normal(2, 0, 4, 64), None, freqs)
    assert a.shape == (2, 0, 4, 64)
    q = normal(4, 2, 64)
    with pytest.raises(GcaError):
        api.rope(q, None, api.rope_freqs(40))
    with pytest.raises(GcaError):
        api.rope(normal(4, 2, 32), None, freqs)
    with pytest.raises(ValueError):
        api.rope(q, None, freqs, positions=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        api.rope(q, None, freqs, positions=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        api.rope(q, None, freqs.cpu())
    with pytest.raises(TypeError):
        api.rope(q.half(), None, freqs)


def test_another_stream_and_a_graph():
    q, k, freqs = normal(2, 100, 4, 64), normal(2, 100, 2, 64, seed=8), api.rope_freqs(64)
    want = api.rope(q, k, freqs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pos = torch.arange(100, dtype=torch.int32, device="cuda").expand(2, 100).contiguous()
    with torch.cuda.stream(s):
        got = api.rope(q, k, freqs, positions=pos)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = api.rope(q, k, freqs, positions=pos)
    pos += 5
    g.replay()
    c, d = api.rope(q, k, freqs, start=5)
    assert torch.equal(a, c) and torch.equal(b, d)


# --- into the paged cache ---------------------------------------------------------------
@pytest.mark.parametrize("qs,kvs,H,Hkv,d,page,rot,inter", [
    ([1], [1], 1, 1, 64, 16, 64, False), ([1] * 40, list(range(1, 400, 10)), 24, 8, 128, 16, 64, True),
    ([5, 0, 130, 1], [300, 7, 130, 64], 6, 2, 64, 64, 32, False), ([7, 3], [4, 100], 2, 1, 64, 32, 64, False),
    ([300], [1000], 12, 12, 64, 128, 64, False), ([2, 2], [50, 60], 128, 2, 128, 16, 128, True)])
def test_append_turns_keys_and_queries(qs, kvs, H, Hkv, d, page, rot, inter):
    g = torch.Generator().manual_seed(sum(kvs))
    T, B = sum(qs), len(qs)
    width = max(-(-n // page) for n in kvs) + 1
    n_pages = B * width + 2
    table = torch.randperm(n_pages, generator=g)[:B * width].view(B, width).to(torch.int32).cuda()
    cu = torch.tensor([0] + qs).cumsum(0).to(torch.int32).cuda()
    kv = torch.tensor(kvs, dtype=torch.int32).cuda()
    x = torch.randn(T + 2, (H + 2 * Hkv) * d, generator=g).to(torch.bfloat16).cuda()       # two rows behind the last sequence
    q, k, v = (y.unflatten(-1, (-1, d)) for y in x.split([H * d, Hkv * d, Hkv * d], -1))
    kc, vc = (torch.randn(n_pages, page, Hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    kc2, vc2 = kc.clone(), vc.clone()
    freqs = api.rope_freqs(rot)
    out = torch.full((T + 2, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = api.paged_rope_append(q, k, v, freqs, kc, vc, table, cu, kv, interleaved=inter, mscale=1.5, out=out)
    assert got is out and api.gca_get_status() == 0
    assert (out[T:] == 7).all()
    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(qs, kvs)])
    check(out[:T], q[:T], freqs, pos, inter, 1.5)
    # the same as the two calls, bit by bit
    a, b = api.rope(q[:T], k[:T], freqs, positions=pos.to(torch.int32).cuda(), interleaved=inter, mscale=1.5)
    assert torch.equal(out[:T], a)
    api.paged_append(b, v[:T].contiguous(), kc2, vc2, table, cu, kv)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_append_bad_pages_and_lengths():
    # a page outside the cache, a table entry of none, lengths that contradict themselves: reported, and
    # nothing else is written
    H = Hkv = 2
    d, page = 64, 16
    table = torch.tensor([[0, 9], [1, -1], [2, 3]], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32).cuda()
    kv = torch.tensor([20, 20, 40], dtype=torch.int32).cuda()
    q, k, v = (normal(3, 2, 64, seed=i) for i in range(3))
    kc, vc = (torch.zeros(4, page, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.full_like(q, 3.0)
    api.paged_rope_append(q, k, v, api.rope_freqs(64), kc, vc, table, cu, kv, out=out)
    assert api.gca_get_status() == 6
    assert (kc == 0).all() and (vc == 0).all()
    assert (out[2] == 3).all() and (out[:2] != 3).any()
    with pytest.raises(ValueError):
        api.paged_rope_append(q, k, v[:2], api.rope_freqs(64), kc, vc, table, cu, kv)
    with pytest.raises(TypeError):
        api.paged_rope_append(q.float(), k, v, api.rope_freqs(64), kc, vc, table, cu, kv)
    with pytest.raises(TypeError):
        api.paged_rope_append(q, k, v, api.rope_freqs(64), kc, vc, table, cu, kv.long())


def test_elements_beyond_32_bits():
    # 2.46e9 elements of q: the last tokens are turned as if they were alone
    T, H, d = 300000, 64, 128
    q = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
    tail = normal(5, H, d, seed=9)
    q[-5:] = tail
    freqs = api.rope_freqs(d)
    api.rope(q, None, freqs, inplace=True)
    want, _ = api.rope(tail, None, freqs, start=T - 5)
    assert torch.equal(q[-5:], want) and not q[:1000].any()
