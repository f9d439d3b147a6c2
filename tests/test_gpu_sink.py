"""Windowed attention with sinks (gca_swa_sink_fwd / _bwd) on the GPU against the
64-bit reference, element by element within the error bounds derived there."""
import pytest
import torch

from retrieval_sparse_attention_gb300 import api
from retrieval_sparse_attention_gb300._lib import GcaError

import sink_reference as ref

pytestmark = pytest.mark.gpu


def inputs(B, L, H, Hkv, d, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(B, L, h, d, generator=g) * std).to(torch.bfloat16) for h in (H, Hkv, Hkv, H)]


def check(q, k, v, dout, window, sinks, scale=0.0, bwd=True):
    qc, kc, vc, gc = (x.cuda() for x in (q, k, v, dout))
    o, lse = api.swa_sink_fwd(qc, kc, vc, window=window, sinks=sinks, attn_scale=scale)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    ro, rl, bo, bl = ref.forward(q, k, v, window, sinks, scale)
    ref.within("o", o, ro, bo)
    ref.within("lse", lse, rl, bl)
    if not bwd:
        return
    grads = api.swa_sink_bwd(qc, kc, vc, o, lse, gc, window=window, sinks=sinks, attn_scale=scale)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    want, bounds = ref.backward(q, k, v, o.cpu(), lse.cpu(), dout, window, sinks, scale)
    for name, a, b, c in zip(("dq", "dk", "dv"), grads, want, bounds):
        ref.within(name, a, b, c)


# (B, L, H, Hkv, d, window, sinks): one token, lengths beside the 128-row tile, windows below,
# at and above it, sinks inside, at and past a tile, sinks beyond the row, groups that do not
# divide the tile, the widest group, no sinks, full causal attention
SHAPES = [(1, 1, 1, 1, 64, 1, 0), (2, 2, 2, 1, 128, 1, 1), (1, 127, 2, 2, 64, 16, 3), (1, 128, 3, 1, 64, 128, 4),
          (2, 129, 4, 2, 128, 100, 1), (1, 517, 6, 2, 64, 64, 4), (1, 700, 2, 2, 128, 129, 16),
          (1, 900, 1, 1, 64, 7, 130), (2, 640, 3, 3, 64, 256, 128), (1, 1000, 6, 2, 64, 200, 1),
          (1, 300, 5, 1, 128, 33, 64), (1, 260, 128, 1, 64, 50, 2), (3, 100, 8, 8, 64, 5000, 4),
          (1, 1100, 2, 1, 128, 512, 0), (1, 200, 4, 4, 64, 1, 0), (1, 400, 7, 1, 64, 1, 500),
          (2, 333, 40, 1, 64, 90, 33), (1, 1300, 2, 2, 64, 1300, 9), (1, 2000, 1, 1, 64, 130, 300)]


@pytest.mark.parametrize("B,L,H,Hkv,d,window,sinks", SHAPES)
def test_every_element(B, L, H, Hkv, d, window, sinks):
    check(*inputs(B, L, H, Hkv, d, seed=L + window), window, sinks)


@pytest.mark.parametrize("d", [64, 128])
def test_large_scores_and_own_scale(d):
    # scores to about +-100: the running maximum moves by far more than any slack a kernel keeps
    q, k, v, g = inputs(1, 600, 4, 2, d, seed=5)
    check(q * 4, k * 4, v, g, 300, 4, scale=1.0 / d ** 0.5)
    check(q, k, v, g, 300, 4, scale=0.01)


def test_rising_scores():
    # every later key scores higher: each tile raises the maximum
    B, L, H, d = 1, 768, 2, 64
    pos = torch.arange(L, dtype=torch.float32).view(1, L, 1, 1)
    q = torch.full((B, L, H, d), 0.5).to(torch.bfloat16)
    k = (pos / 16.0 * torch.ones(B, L, H, d)).to(torch.bfloat16)
    _, _, v, g = inputs(B, L, H, H, d, seed=2)
    check(q, k, v, g, 512, 4)
    check(q, -k, v, g, 512, 4)           # and the sinks above all others


def test_packed_projection():
    # q, k, v as slices of one projection's output: token strides, one shared key head
    B, L, H, Hkv, d = 2, 300, 4, 2, 64
    g = torch.Generator().manual_seed(9)
    x = torch.randn(B, L, (H + 2 * Hkv) * d, generator=g).to(torch.bfloat16)
    dout = torch.randn(B, L, H, d, generator=g).to(torch.bfloat16)

    def parts(x):
        a, b, c = x.split([H * d, Hkv * d, Hkv * d], -1)
        return a.unflatten(-1, (H, d)), b.unflatten(-1, (Hkv, d)), c.unflatten(-1, (Hkv, d))
    xc = x.cuda()
    q, k, v = parts(xc)
    assert not q.is_contiguous()
    o, lse = api.swa_sink_fwd(q, k, v, window=100, sinks=4)
    grads = api.swa_sink_bwd(q, k, v, o, lse, dout.cuda(), window=100, sinks=4)
    o2, lse2 = api.swa_sink_fwd(*(t.contiguous() for t in (q, k, v)), window=100, sinks=4)
    grads2 = api.swa_sink_bwd(*(t.contiguous() for t in (q, k, v)), o, lse, dout.cuda(), window=100, sinks=4)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(grads, grads2))
    ro, rl, bo, bl = ref.forward(*parts(x), 100, 4)
    ref.within("o", o, ro, bo)
    ref.within("lse", lse, rl, bl)


def test_agrees_with_the_plain_window():
    # without sinks this is the sliding-window operator that the library has had
    q, k, v, g = (x.cuda() for x in inputs(2, 1024, 3, 3, 64, seed=4))
    o, lse = api.swa_sink_fwd(q, k, v, window=512, sinks=0)
    o2, lse2 = api.swa_fwd(q, k, v, window=512)
    _, _, bo, bl = ref.forward(q.cpu(), k.cpu(), v.cpu(), 512, 0)
    ref.within("o", o, o2.double().cpu(), 2 * bo)
    ref.within("lse", lse, lse2.double().cpu(), 2 * bl)


def test_padded_batch():
    # rows behind a sequence's end: masked out by dout = 0, they leave no gradient behind,
    # and the rows before them do not see them
    q, k, v, g = inputs(1, 400, 2, 1, 64, seed=6)
    n = 250
    g[:, n:] = 0
    qc, kc, vc, gc = (x.cuda() for x in (q, k, v, g))
    o, lse = api.swa_sink_fwd(qc, kc, vc, window=90, sinks=4)
    dq, dk, dv = api.swa_sink_bwd(qc, kc, vc, o, lse, gc, window=90, sinks=4)
    for x in (dk, dv):
        assert (x[:, n:] == 0).all()
    qs, ks, vs, gs = (x[:, :n] for x in (q, k, v, g))
    ro, rl, bo, bl = ref.forward(qs, ks, vs, 90, 4)
    ref.within("o", o[:, :n], ro, bo)
    want, bounds = ref.backward(qs, ks, vs, o[:, :n].cpu(), lse[:, :n].cpu(), gs, 90, 4)
    # (the last row's accumulation bound covers the zero terms too)
    for a, b, c in zip((dq, dk, dv), want, bounds):
        ref.within("grad", a[:, :n], b, c)


def test_deterministic_and_fully_written():
    q, k, v, g = (x.cuda() for x in inputs(2, 1500, 6, 2, 64, seed=5))
    a = api.swa_sink_fwd(q, k, v, window=300, sinks=4)
    ga = api.swa_sink_bwd(q, k, v, *a, g, window=300, sinks=4)
    p = api.make_swa_sink_params(B=2, L=1500, H=6, Hkv=2, d=64, window=300, sinks=4)
    for fill in (float("nan"), 7.0):
        o, lse = torch.full_like(q, fill), torch.full(q.shape[:3], fill, device="cuda")
        ws = torch.full((api.gca_swa_sink_fwd_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
        api.gca_swa_sink_fwd(p, q, k, v, o, lse, ws)
        assert torch.equal(o, a[0]) and torch.equal(lse, a[1])
        dq, dk, dv = torch.full_like(q, fill), torch.full_like(k, fill), torch.full_like(v, fill)
        ws = torch.full((api.gca_swa_sink_bwd_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
        api.gca_swa_sink_bwd(p, q, k, v, o, lse, g, dq, dk, dv, ws)
        assert all(torch.equal(x, y) for x, y in zip((dq, dk, dv), ga))
    assert api.gca_get_status() == 0


def test_a_workspace_of_256_bytes_stays_untouched():
    q, k, v, _ = (x.cuda() for x in inputs(1, 900, 6, 2, 64, seed=15))
    p = api.make_swa_sink_params(B=1, L=900, H=6, Hkv=2, d=64, window=200, sinks=4)
    assert api.gca_swa_sink_fwd_workspace_size(p) == 256
    want = api.swa_sink_fwd(q, k, v, window=200, sinks=4)
    ws = torch.full((256,), 77, dtype=torch.uint8, device="cuda")
    got = api.swa_sink_fwd(q, k, v, window=200, sinks=4, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and (ws == 77).all()
    assert api.gca_last_launch_count() == 1


def test_other_stream_and_graph():
    q, k, v, g = (x.cuda() for x in inputs(1, 700, 4, 2, 64, seed=8))
    want = api.swa_sink_fwd(q, k, v, window=200, sinks=4)
    gw = api.swa_sink_bwd(q, k, v, *want, g, window=200, sinks=4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = api.swa_sink_fwd(q, k, v, window=200, sinks=4)
        gg = api.swa_sink_bwd(q, k, v, *got, g, window=200, sinks=4)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want + gw, got + gg))
    q2 = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = api.swa_sink_fwd(q2, k, v, window=200, sinks=4)
        gg = api.swa_sink_bwd(q2, k, v, *got, g, window=200, sinks=4)
    for src in (q, q.flip(1).contiguous(), q):
        q2.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want + gw, got + gg))


def test_two_streams_at_once():
    # calls that overlap, each with its own workspace, against the same calls one after the other
    a = [x.cuda() for x in inputs(4, 2000, 6, 2, 64, seed=10)]
    b = [x.cuda() for x in inputs(1, 5000, 8, 2, 128, seed=11)]

    def step(t, window, sinks):
        o, lse = api.swa_sink_fwd(*t[:3], window=window, sinks=sinks)
        return (o, lse) + api.swa_sink_bwd(*t[:3], o, lse, t[3], window=window, sinks=sinks)

    want = step(a, 512, 4) + step(b, 900, 16)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(6):
        with torch.cuda.stream(sa):
            ga = step(a, 512, 4)
        with torch.cuda.stream(sb):
            gb = step(b, 900, 16)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ga + gb, want))
    assert api.gca_get_status() == 0


def test_graphs_that_share_a_workspace():
    # two captured calls of different shapes over one workspace, replayed in turn on one stream
    a = [x.cuda() for x in inputs(1, 3000, 4, 2, 64, seed=12)]
    b = [x.cuda() for x in inputs(2, 900, 8, 1, 128, seed=13)]
    want = api.swa_sink_fwd(*a[:3], window=700, sinks=4) + api.swa_sink_fwd(*b[:3], window=300, sinks=1)
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for t, window, sinks in ((a, 700, 4), (b, 300, 1)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.extend(api.swa_sink_fwd(*t[:3], window=window, sinks=sinks, workspace=ws))
    for _ in range(3):
        for x in got:
            x.zero_()
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert api.gca_get_status() == 0


# enough key tiles for shares of many units, whole and cut, and for a sink's long item to be
# spread over many shares; the 64-bit reference on the GPU
@pytest.mark.parametrize("B,L,H,Hkv,d,window,sinks", [(2, 4000, 12, 12, 64, 512, 4), (2, 3001, 8, 2, 128, 700, 16),
                                                      (1, 5003, 6, 1, 64, 1200, 40), (3, 2500, 5, 5, 128, 130, 1),
                                                      (1, 6000, 4, 2, 64, 6000, 0), (5, 1900, 9, 3, 64, 257, 200)])
def test_every_element_of_longer_rows(B, L, H, Hkv, d, window, sinks):
    q, k, v, g = (x.cuda() for x in inputs(B, L, H, Hkv, d, seed=L))
    o, lse = api.swa_sink_fwd(q, k, v, window=window, sinks=sinks)
    grads = api.swa_sink_bwd(q, k, v, o, lse, g, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    for b in range(B):
        one = slice(b, b + 1)
        ro, rl, bo, bl = ref.forward(q[one], k[one], v[one], window, sinks)
        ref.within("o", o[one], ro.cpu(), bo.cpu())
        ref.within("lse", lse[one], rl.cpu(), bl.cpu())
        del ro, rl, bo, bl
        want, bounds = ref.backward(q[one], k[one], v[one], o[one], lse[one], g[one], window, sinks)
        for name, a, w, c in zip(("dq", "dk", "dv"), grads, want, bounds):
            ref.within(name, a[one], w.cpu(), c.cpu())
        del want, bounds
    torch.cuda.empty_cache()


# a few units more than there are workers, of many tiles each: windows whose units are cut
@pytest.mark.parametrize("B,L,H,Hkv,d,window,sinks", [(1, 3300, 12, 12, 64, 1500, 4), (1, 2464, 16, 4, 128, 1800, 16),
                                                      (1, 3290, 12, 12, 64, 2000, 0)])
def test_windows_whose_units_are_cut(B, L, H, Hkv, d, window, sinks):
    test_every_element_of_longer_rows(B, L, H, Hkv, d, window, sinks)


def test_full_size_sampled():
    # the 12-head model's batch: single rows against the reference on what they see
    B, L, H, d, W, ns = 8, 16384, 12, 64, 512, 4
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, g = (torch.randn(B, L, H, d, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(4))
    o, lse = api.swa_sink_fwd(q, k, v, window=W, sinks=ns)
    dq, dk, dv = api.swa_sink_bwd(q, k, v, o, lse, g, window=W, sinks=ns)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    rng = torch.Generator().manual_seed(1)
    some = [(int(torch.randint(B, (1,), generator=rng)), int(torch.randint(L, (1,), generator=rng))) for _ in range(40)]
    for b, t in [(0, 0), (7, L - 1), (3, 511), (3, 515), (5, 128), (2, 9999), (6, 4097)] + some:
        kpos = torch.cat([torch.arange(min(ns, max(0, t - W + 1))), torch.arange(max(0, t - W + 1), t + 1)])
        qpos = torch.tensor([t])
        kk, vv = k[b].cpu()[kpos], v[b].cpu()[kpos]
        ro, rl, bo, bl = ref.rows(q[b, t:t + 1].cpu(), kk, vv, qpos, kpos, W, ns)
        ref.within("o", o[b, t:t + 1], ro, bo)
        ref.within("lse", lse[b, t:t + 1], rl, bl)
        p = torch.exp(torch.einsum("hd,shd->hs", q[b, t].double().cpu(), kk.double()) * d ** -0.5
                      - lse[b, t].double().cpu()[:, None])
        dl = (g[b, t].double() * o[b, t].double()).sum(-1).cpu()
        ds = p * (torch.einsum("hd,shd->hs", g[b, t].double().cpu(), vv.double()) - dl[:, None]) * d ** -0.5
        want = torch.einsum("hs,shd->hd", ds, kk.double())
        bound = (2 ** -8 + 2 ** -11) * (torch.einsum("hs,shd->hd", ds.abs(), kk.double().abs()) + want.abs()) + 1e-4
        ref.within("dq", dq[b, t], want, bound)
    # the sinks' gradients gather from every query of the row; a late key's from its window only
    for b, s in [(1, 0), (4, 3), (2, 4), (0, 16000)]:
        last = L if s < ns else min(L, s + W)
        qq, gg, oo, ll = (x[b, s:last].double() for x in (q, g, o, lse))
        p = torch.exp(torch.einsum("thd,hd->ht", qq, k[b, s].double()) * d ** -0.5 - ll.t())
        dp = torch.einsum("thd,hd->ht", gg, v[b, s].double())
        ds = p * (dp - (gg * oo).sum(-1).t()) * d ** -0.5
        for name, got, w, x in (("dk", dk, ds, qq), ("dv", dv, p, gg)):
            want = torch.einsum("ht,thd->hd", w, x)
            mag = torch.einsum("ht,thd->hd", w.abs(), x.abs())
            ref.within(name, got[b, s], want.cpu(), ((2 ** -8 + 2 ** -10) * (mag + want.abs()) + 1e-4).cpu())


def test_refusals():
    q, k, v, g = (x.cuda() for x in inputs(1, 64, 4, 2, 64, seed=1))
    with pytest.raises(GcaError) as e:
        api.swa_sink_fwd(q.float(), k.float(), v.float(), window=8, sinks=1)
    assert e.value.code == 2
    with pytest.raises(TypeError):
        api.swa_sink_fwd(q, k.float(), v, window=8, sinks=1)
    with pytest.raises(ValueError):
        api.swa_sink_fwd(q, k[:, :32], v[:, :32], window=8, sinks=1)
    with pytest.raises(ValueError):
        api.swa_sink_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, window=8, sinks=1)
    with pytest.raises(ValueError):
        api.swa_sink_fwd(q[:, :1].expand(1, 64, 4, 64), k, v, window=8, sinks=1)
    with pytest.raises(GcaError) as e:
        api.swa_sink_fwd(q, k, v, window=0, sinks=1)
    assert e.value.code == 1
    o, lse = api.swa_sink_fwd(q, k, v, window=8, sinks=1)
    with pytest.raises(ValueError):
        api.swa_sink_bwd(q, k, v, o, lse[:, :32], g, window=8, sinks=1)
    with pytest.raises(TypeError):
        api.swa_sink_bwd(q, k, v, o, lse.half(), g, window=8, sinks=1)
    with pytest.raises(GcaError) as e:
        api.swa_sink_fwd(q, k, v, window=8, sinks=1, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 3
