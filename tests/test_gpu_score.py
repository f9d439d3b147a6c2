"""Windowed attention with capped or biased scores on the GPU, dense with gradients and over the
paged cache, against the 64-bit reference, element by element within the bounds derived there."""
import pytest
import torch

from retrieval_sparse_attention_gb300 import api
from retrieval_sparse_attention_gb300._lib import GcaError

import score_reference as ref
from test_gpu_paged import Cache
from test_gpu_sink import inputs

pytestmark = pytest.mark.gpu


def slopes_of(H, kind="usual"):
    i = torch.arange(1, H + 1, dtype=torch.float32)
    return {"usual": 2.0 ** (-8 * i / H), "steep": 8.0 / i, "rising": -0.01 * i, "none": torch.zeros(H)}[kind]


def check(q, k, v, dout, window, sinks, cap=0.0, slopes=None, scale=0.0):
    qc, kc, vc, gc = (x.cuda() for x in (q, k, v, dout))
    kw = dict(window=window, sinks=sinks, attn_scale=scale, softcap=cap, slopes=None if slopes is None else slopes.cuda())
    o, lse = api.swa_sink_fwd(qc, kc, vc, **kw)
    grads = api.swa_sink_bwd(qc, kc, vc, o, lse, gc, **kw)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    ro, rl, bo, bl = ref.forward(q, k, v, window, sinks, cap, slopes, scale)
    ref.within("o", o, ro, bo)
    ref.within("lse", lse, rl, bl)
    want, bounds = ref.backward(q, k, v, o.cpu(), lse.cpu(), dout, window, sinks, cap, slopes, scale)
    for name, a, b, c in zip(("dq", "dk", "dv"), grads, want, bounds):
        ref.within(name, a, b, c)
    return o, lse, grads


# one token, lengths beside the tiles, windows below, at and above one, sinks inside, at and past a
# tile (narrow tiles up to 32 sinks), groups that do not divide the tile, full causal attention
SHAPES = [(1, 1, 1, 1, 64, 1, 0), (2, 129, 4, 2, 128, 100, 1), (1, 517, 6, 2, 64, 64, 4), (1, 700, 2, 2, 128, 129, 16),
          (1, 900, 1, 1, 64, 7, 130), (1, 300, 5, 1, 128, 33, 64), (1, 260, 128, 1, 64, 50, 2), (3, 100, 8, 8, 64, 5000, 4),
          (1, 400, 7, 1, 64, 1, 500), (2, 333, 40, 1, 64, 90, 33), (1, 1300, 2, 2, 64, 512, 9), (1, 1100, 2, 1, 128, 512, 0)]


@pytest.mark.parametrize("B,L,H,Hkv,d,window,sinks", SHAPES)
@pytest.mark.parametrize("cap,kind", [(3.0, None), (50.0, None), (0.0, "usual"), (0.0, "steep")])
def test_every_element(B, L, H, Hkv, d, window, sinks, cap, kind):
    q, k, v, g = inputs(B, L, H, Hkv, d, seed=L + window)
    check(q * 2, k, v, g, window, sinks, cap, slopes_of(H, kind) if kind else None)


@pytest.mark.parametrize("d", [64, 128])
def test_scores_far_beyond_the_cap(d):
    # products to about +-100 under a cap of 20, and a cap so wide that it hardly shows
    q, k, v, g = inputs(1, 600, 4, 2, d, seed=5)
    check(q * 4, k * 4, v, g, 300, 4, 20.0)
    check(q * 4, k * 4, v, g, 300, 4, 1024.0)
    check(q, k, v, g, 300, 4, 2.0 ** -10)


@pytest.mark.parametrize("cap", [30.0, 51.9, 52.1])
def test_scores_at_either_cap(cap):
    # rows whose scores all lie near -cap, and near +cap, with small and large values: on either side of
    # the largest cap that is taken against a fixed maximum (51.98)
    g = torch.Generator().manual_seed(17)
    L, d = 300, 64
    u = torch.sign(torch.randn(1, 1, 1, d, generator=g))
    k = (u * 2 + 0.1 * torch.randn(1, L, 1, d, generator=g)).to(torch.bfloat16)
    q = torch.cat([-8 * u.expand(1, L, 1, d), 8 * u.expand(1, L, 1, d)], 2)
    q = (q + 0.1 * torch.randn(1, L, 2, d, generator=g)).to(torch.bfloat16)
    v = torch.randn(1, L, 1, d, generator=g)
    v[..., :20] *= 2.0 ** -40
    v[..., 20:40] *= 2.0 ** 33
    v = v.to(torch.bfloat16)
    dout = torch.randn(1, L, 2, d, generator=g).to(torch.bfloat16)
    kw = dict(window=120, sinks=3, softcap=cap)
    o, lse = api.swa_sink_fwd(q.cuda(), k.cuda(), v.cuda(), **kw)
    ro, rl, bo, bl = ref.forward(q, k, v, 120, 3, cap)
    ref.within("o", o, ro, bo)
    ref.within("lse", lse, rl, bl)
    assert lse[0, :, 0].max() < -0.6 * cap and lse[0, :, 1].min() > 0.6 * cap
    check(q, k, v.clamp(-4, 4), dout, 120, 3, cap)


def test_a_scale_of_its_own():
    q, k, v, g = inputs(2, 300, 4, 2, 64, seed=14)
    check(q, k, v, g, 100, 4, 6.0, scale=0.4)
    check(q, k, v, g, 100, 4, 0.0, slopes_of(4), scale=0.03)


def test_infinite_products_count_as_the_cap():
    # (1e38 x 64 keys of 1e2 overflow fp32: the tanh of either is the same number)
    q, k, v, g = inputs(1, 300, 2, 2, 64, seed=8)
    q[0, 100] = 1e38 * torch.sign(q[0, 100])
    k[0, :, 0, 0] = 100.0 * torch.sign(k[0, :, 0, 0])
    q[0, 100, 1] = 1.0
    q[0, 100, 0, 1:] = 0.0                       # (one term a product: +inf or -inf, never their sum)
    k[0, :, 0, 1:] = k[0, :, 0, 1:].clamp(-4, 4)
    kw = dict(window=128, sinks=2, softcap=10.0)
    o, lse = api.swa_sink_fwd(q.cuda(), k.cuda(), v.cuda(), **kw)
    ro, rl, bo, bl = ref.forward(q, k, v, 128, 2, 10.0)
    rest = [i for i in range(300) if i != 100]
    ref.within("o", o[:, rest], ro[:, rest], bo[:, rest])
    # row 100 of head 0 has products whose error bound is of no use: the scores are +-10 all the same
    s = 10.0 * torch.sign(q[0, 100, 0, 0].double() * k[0, :, 0, 0].double())
    see = torch.zeros(300, dtype=torch.bool)
    see[:101] = True
    p = torch.softmax(s.masked_fill(~see, float("-inf")), 0)
    want = p @ v[0, :, 0].double()
    bound = 2.0 ** -8 * (want.abs() + p @ v[0, :, 0].double().abs()) * 1.01 + 2.0 ** -18
    assert ((o[0, 100, 0].double().cpu() - want).abs() <= bound).all()


@pytest.mark.parametrize("kind", ["rising", "none"])
def test_other_slopes(kind):
    q, k, v, g = inputs(2, 500, 4, 2, 64, seed=6)
    check(q, k, v, g, 130, 40, 0.0, slopes_of(4, kind))


def test_no_slope_is_the_plain_attention():
    q, k, v, g = (x.cuda() for x in inputs(1, 700, 4, 2, 64, seed=7))
    a, la = api.swa_sink_fwd(q, k, v, window=200, sinks=4)
    b, lb = api.swa_sink_fwd(q, k, v, window=200, sinks=4, slopes=torch.zeros(4, device="cuda"))
    # the same sums from scores rounded once more (2^-24 of a few units each), and bf16 outputs that may
    # fall on either side of a border
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -8 * a.float().abs().max()
    assert (la - lb).abs().max() <= 1e-5


def test_falling_bias_over_long_rows():
    # sinks tens of thousands of tokens back: their bias is thousands of units, the near keys' a few
    B, L, H, d, W, ns = 1, 20000, 2, 64, 256, 40
    q, k, v, g = inputs(B, L, H, H, d, seed=11)
    slopes = torch.tensor([0.25, 1e-4])
    o, lse = api.swa_sink_fwd(q.cuda(), k.cuda(), v.cuda(), window=W, sinks=ns, slopes=slopes.cuda())
    assert api.gca_get_status() == 0
    for r0 in (0, 5000, L - 130):
        r = torch.arange(r0, r0 + 130)
        kp = torch.cat([torch.arange(min(ns, max(0, r0 - W + 1))), torch.arange(max(0, r0 - W + 1), r0 + 130)])
        ro, rl, bo, bl = ref.rows(q[0, r], k[0, kp], v[0, kp], r, kp, W, ns, 0.0, slopes)
        ref.within("o", o[0, r], ro, bo)
        ref.within("lse", lse[0, r], rl, bl)


@pytest.mark.parametrize("cap,bias", [(15.0, False), (0.0, True)])
def test_units_cut_and_joined(cap, bias):
    # few long rows: units shared by several CTAs, partial sums joined; equal bit by bit from run to run
    q, k, v, g = inputs(1, 1500, 4, 1, 128, seed=12)
    slopes = slopes_of(4) if bias else None
    a = check(q, k, v, g, 1500, 0, cap, slopes)
    b = check(q, k, v, g, 1500, 0, cap, slopes)
    assert torch.equal(a[0], b[0]) and all(torch.equal(x, y) for x, y in zip(a[2], b[2]))


def test_packed_projection():
    B, L, H, Hkv, d = 2, 300, 4, 2, 64
    g = torch.Generator().manual_seed(9)
    x = torch.randn(B, L, (H + 2 * Hkv) * d, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (y.unflatten(-1, (-1, d)) for y in x.split([H * d, Hkv * d, Hkv * d], -1))
    dense = [y.contiguous() for y in (q, k, v)]
    for kw in (dict(softcap=4.0), dict(slopes=slopes_of(H).cuda())):
        a = api.swa_sink_fwd(q, k, v, window=90, sinks=3, **kw)
        b = api.swa_sink_fwd(*dense, window=90, sinks=3, **kw)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


PAGED = [([1], [1], 1, 1, 64, 16, 0, 0), ([1], [777], 12, 12, 64, 64, 512, 4), ([1, 0, 3, 40, 0, 1], [300, 50, 3, 100, 0, 17], 6, 2, 64, 16, 64, 4),
         ([130, 1, 257], [130, 1000, 700], 4, 4, 64, 128, 0, 0), ([200], [900], 8, 1, 128, 64, 100, 16),
         ([33, 5], [33, 4000], 3, 1, 64, 64, 129, 33), ([1] * 20, list(range(1, 400, 20)), 8, 1, 64, 16, 0, 0),
         ([2, 1], [600, 601], 128, 1, 64, 32, 30, 1), ([1, 3, 1], [30000, 9000, 70], 4, 2, 128, 64, 0, 0),
         ([5, 4], [3, 0], 2, 1, 64, 16, 0, 0),
         # units of eight rows and less: chunks of a few tokens, groups that do not divide eight
         ([2, 4, 8, 3], [40, 700, 130, 129], 4, 4, 64, 16, 100, 3), ([2, 4, 1, 3], [600, 5, 257, 128], 4, 2, 128, 64, 0, 0),
         ([2, 1, 2], [3000, 200, 131], 6, 2, 64, 32, 130, 40), ([1, 1], [500, 20], 5, 1, 128, 16, 33, 1)]


@pytest.mark.parametrize("qs,kvs,H,Hkv,d,page,window,sinks", PAGED)
@pytest.mark.parametrize("cap", [7.0, 0.0])
def test_over_the_paged_cache(qs, kvs, H, Hkv, d, page, window, sinks, cap):
    c = Cache(qs, kvs, H, Hkv, d, page, seed=sum(kvs))
    slopes = None if cap else slopes_of(H)
    o, lse = api.paged_attn(*c.cuda(), max_q=max(qs), window=window, sinks=sinks, with_lse=True, softcap=cap,
                            slopes=None if cap else slopes.cuda())
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    for b, (n, kv) in enumerate(zip(qs, kvs)):
        if n == 0:
            continue
        at = slice(int(c.cu[b]), int(c.cu[b + 1]))
        if kv == 0:                                # tokens before the first position see nothing
            assert (o[at] == 0).all() and torch.isneginf(lse[at]).all()
            continue
        ro, rl, bo, bl = ref.rows(c.q[at], c.k[b], c.v[b], torch.arange(kv - n, kv), torch.arange(kv), window, sinks, cap, slopes)
        ref.within("o of sequence %d" % b, o[at], ro, bo)
        ref.within("lse of sequence %d" % b, lse[at], rl, bl)


def test_a_captured_step_follows_lengths_and_slopes():
    c = Cache([1, 1], [200, 900], 4, 2, 64, 16, seed=3)
    q, kc, vc, table, cu, kv = c.cuda()
    kc, vc = kc.nan_to_num(0.0), vc.nan_to_num(0.0)
    slopes = slopes_of(4).cuda()
    kw = dict(max_q=1, window=300, sinks=2, with_lse=True, slopes=slopes)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.paged_attn(q, kc, vc, table, cu, kv, out=out, **kw)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, lse = api.paged_attn(q, kc, vc, table, cu, kv, out=out, **kw)
    for n, f in ((150, 1.0), (180, 3.0)):
        kv[0] = n
        slopes.mul_(f)
        g.replay()
        want, want_lse = api.paged_attn(q, kc, vc, table, cu, kv, **kw)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_refusals():
    q, k, v, g = (x.cuda() for x in inputs(1, 64, 2, 2, 64, seed=1))
    with pytest.raises(GcaError):
        api.swa_sink_fwd(q, k, v, window=8, sinks=0, softcap=5.0, slopes=torch.ones(2, device="cuda"))
    with pytest.raises(GcaError):
        api.swa_sink_fwd(q, k, v, window=8, sinks=0, softcap=float("nan"))
    with pytest.raises(ValueError):
        api.swa_sink_fwd(q, k, v, window=8, sinks=0, slopes=torch.ones(2))
    with pytest.raises(ValueError):
        api.swa_sink_fwd(q, k, v, window=8, sinks=0, slopes=torch.ones(3, device="cuda"))


@pytest.mark.parametrize("cap,bias", [(9.0, False), (0.0, True)])
def test_training_step_captured_and_on_another_stream(cap, bias):
    # (a workspace that the caller keeps, units cut and joined in both passes)
    q, k, v, g = (x.cuda() for x in inputs(2, 700, 8, 2, 64, seed=21))
    kw = dict(window=300, sinks=3, softcap=cap, slopes=slopes_of(8).cuda() if bias else None)
    p = api.make_swa_sink_params(B=2, L=700, H=8, Hkv=2, d=64, window=300, sinks=3)
    ws = torch.empty(api.gca_swa_sink_bwd_scored_workspace_size(p), dtype=torch.uint8, device="cuda")
    assert ws.numel() > api.gca_swa_sink_bwd_workspace_size(p)

    def step():
        o, lse = api.swa_sink_fwd(q, k, v, **kw)
        return [o, lse, *api.swa_sink_bwd(q, k, v, o, lse, g, workspace=ws, **kw)]
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    q.mul_(0.5)
    graph.replay()
    held = [x.clone() for x in got]
    assert not torch.equal(held[0], want[0])
    ws.fill_(255)                                # (what a workspace held before does not matter)
    assert all(torch.equal(a, b) for a, b in zip(held, step()))
    assert api.gca_get_status() == 0


def test_gradients_need_their_own_workspace():
    q, k, v, g = (x.cuda() for x in inputs(1, 200, 2, 2, 64, seed=22))
    kw = dict(window=50, sinks=0, softcap=5.0)
    o, lse = api.swa_sink_fwd(q, k, v, **kw)
    p = api.make_swa_sink_params(B=1, L=200, H=2, d=64, window=50)
    small = torch.empty(api.gca_swa_sink_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    with pytest.raises(GcaError) as e:
        api.swa_sink_bwd(q, k, v, o, lse, g, workspace=small, **kw)
    assert e.value.code == 3


def test_rows_of_a_few_keys():
    # 16 tokens, scores of several units: dP - delta is a difference of near numbers.  The roundings of the
    # result and of ds are 1.7e-3 of the norm each (uniform within half a step of bf16, relative to a
    # value anywhere between two powers of two), 2.4e-3 together; an eighth more for so few values
    for cap, slopes in ((0.0, slopes_of(6)), (50.0, None), (3.0, None)):
        q, k, v, g = inputs(4, 16, 6, 2, 64, seed=23)
        q = q * 3
        kw = dict(window=16, sinks=1, softcap=cap, slopes=None if slopes is None else slopes.cuda())
        x = [t.cuda() for t in (q, k, v)]
        o, lse = api.swa_sink_fwd(*x, **kw)
        got = api.swa_sink_bwd(*x, o, lse, g.cuda(), **kw)
        ro, rl, _, _ = ref.forward(q, k, v, 16, 1, cap, slopes)
        want, _ = ref.backward(q, k, v, ro, rl, g, 16, 1, cap, slopes)
        for a, b in zip(got[:2], want[:2]):
            assert float((a.double().cpu() - b).norm() / b.norm()) <= 2.7e-3
