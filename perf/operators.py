"""Timed cases of the windowed attention with sinks and of the attention over a paged K/V cache.

Four operators: the attention of a sequence over a sliding window and a few
first tokens that stay visible (sinks), forward for prompts and forward plus
gradients for training; the write of new tokens into a paged K/V cache; and
the attention of new tokens (one each, or a chunk) over that cache.

``run`` computes an operator in plain 32-bit torch operations, or, where
``own`` is true, by the calls a user makes of this package.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_BLOCK = 256          # queries that the plain form takes together


# --- cases ------------------------------------------------------------------------------
def listed():
    return [
        # one short prompt: a few tiles in all, the time of the launches counts
        dict(name="fwd_b1_517", kind="fwd", B=1, L=517, H=12, Hkv=12, d=64, window=128, sinks=4),
        # prompts of the 12-head model: the shape of its training batch
        dict(name="fwd_b8_16k", kind="fwd", B=8, L=16384, H=12, Hkv=12, d=64, window=512, sinks=4),
        # one long prompt with shared key heads
        dict(name="fwd_b1_64k_shared", kind="fwd", B=1, L=65536, H=16, Hkv=4, d=128, window=1024, sinks=16),
        # a training step on short odd sequences, three query heads to a key head
        dict(name="train_b3_1000", kind="train", B=3, L=1000, H=6, Hkv=2, d=64, window=200, sinks=1),
        # a training step of the 12-head model at its own batch
        dict(name="train_b8_16k", kind="train", B=8, L=16384, H=12, Hkv=12, d=64, window=512, sinks=4),
        # a training step with shared key heads and the wider head
        dict(name="train_b2_16k_shared", kind="train", B=2, L=16384, H=16, Hkv=4, d=128, window=1024, sinks=16),
        # the write of one generated token of each of 64 requests
        dict(name="append_b64_tokens", kind="append", B=64, q_max=1, q_min=1, kv_max=4096, kv_min=64, ragged=1,
             H=8, Hkv=8, d=128, page=64, window=0, sinks=0),
        # the write of eight prompt chunks of uneven length
        dict(name="append_b8_chunks", kind="append", B=8, q_max=2048, q_min=900, kv_max=8192, kv_min=2048, ragged=2,
             H=12, Hkv=12, d=64, page=64, window=0, sinks=0),
        # one token of one request through the window: latency
        dict(name="paged_b1_token", kind="paged", B=1, q_max=1, q_min=1, kv_max=777, kv_min=777, ragged=3,
             H=12, Hkv=12, d=64, page=64, window=512, sinks=4),
        # one token of each of 32 long requests over their whole caches: bound by the cache's bytes
        dict(name="paged_b32_tokens_32k", kind="paged", B=32, q_max=1, q_min=1, kv_max=32768, kv_min=4096, ragged=4,
             H=24, Hkv=8, d=128, page=64, window=0, sinks=0),
        # chunks of four long prompts over the whole cache so far: bound by the products
        dict(name="paged_b4_chunks_16k", kind="paged", B=4, q_max=2048, q_min=1500, kv_max=16384, kv_min=6000, ragged=5,
             H=16, Hkv=4, d=128, page=64, window=0, sinks=0),
        # a serving batch: idle slots, single tokens and prompt chunks together, through the window
        dict(name="paged_b48_mixed", kind="paged", B=48, q_max=512, q_min=0, kv_max=6000, kv_min=512, ragged=6,
             H=12, Hkv=12, d=64, page=16, window=512, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["fwd", "train", "append", "paged", "paged"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 12])
    H = Hkv * rng.choice([1, 2, 3, 4, 8] if Hkv <= 4 else [1, 2, 3])
    sinks = rng.choice([0, 1, 4, 16, 33, 64])
    if kind in ("fwd", "train"):
        # (a training sequence has some tokens: the first one's query gradient is zero whatever the inputs)
        least = 1 if kind == "fwd" else 16
        B, L, W = _log_int(rng, 1, 8), _log_int(rng, least, 32768), _log_int(rng, 16, 2048)
        while B * L * H * d * (W + sinks + 128) > 2.5e10:      # under half the largest listed one
            L = max(least, L // 2 + rng.randrange(3))
            B = max(1, B - 1)
        return dict(kind=kind, B=B, L=L, H=H, Hkv=Hkv, d=d, window=W, sinks=sinks)
    page = rng.choice([16, 32, 64, 128])
    B = _log_int(rng, 1, 64)
    q_max = rng.choice([1, 1, _log_int(rng, 2, 2048)])
    kv_max = max(q_max, _log_int(rng, 16, 32768))
    while B * q_max * kv_max * H * d > 1.2e11 or B * kv_max * Hkv * d > 5e8:
        kv_max = max(16, kv_max // 2 + rng.randrange(5))
        q_max = min(q_max, kv_max)
        B = max(1, B * 3 // 4)
    q_min = 1 if q_max == 1 else rng.choice([0, 1, q_max])
    kv_min = max(q_max, kv_max // rng.choice([1, 4, 20]))
    window = rng.choice([0, _log_int(rng, 16, 4096)])
    return dict(kind=kind, B=B, q_max=q_max, q_min=q_min, kv_max=max(kv_max, kv_min), kv_min=kv_min,
                ragged=rng.randrange(1 << 20), H=H, Hkv=Hkv, d=d, page=page, window=window,
                sinks=sinks if window else 0)


def _lengths(c):
    """New tokens and cached tokens (the new ones included) of each sequence of a paged case."""
    r = random.Random(c["ragged"])
    qs, kvs = [], []
    for i in range(c["B"]):
        # a wide range of new tokens is a serving batch: half of its slots hold one token, an eighth none
        wide = c["q_max"] > 16 and c["q_min"] <= 1
        u = r.random()
        if i == 0:
            n = c["q_max"]
        elif wide and u < 0.625:
            n = 1 if u < 0.5 or c["q_min"] == 1 else 0
        else:
            n = r.randint(c["q_min"], c["q_max"])
        qs.append(n)
        kvs.append(max(n, c["kv_max"] if i == 0 else r.randint(c["kv_min"], c["kv_max"])))
    return qs, kvs


def _pairs(c):
    """(query, visible key) pairs of one query head."""
    W, ns = c["window"], c["sinks"]
    if c["kind"] in ("fwd", "train"):
        spans = [(0, c["L"])] * c["B"]
    else:
        spans = [(kv - q, kv) for q, kv in zip(*_lengths(c))]

    def upto(n):                       # sum over positions p < n of the keys that p sees
        if not W:
            return n * (n + 1) // 2
        a = min(n, W)
        total = a * (a + 1) // 2 + (n - a) * W
        b = max(0, min(n - W, ns))     # the first sinks to leave the window, one by one
        return total + b * (b + 1) // 2 + max(0, n - W - b) * b
    return sum(upto(hi) - upto(lo) for lo, hi in spans)


def work(case):
    c = case
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    if c["kind"] in ("fwd", "train"):
        tok, pairs = c["B"] * c["L"], _pairs(c) * H
        byt = 2 * tok * (2 * H + 2 * Hkv) * d + 4 * tok * H
        if c["kind"] == "fwd":
            return dict(bytes=byt, flops=4 * d * pairs)
        return dict(bytes=byt + 2 * tok * (2 * H + 2 * Hkv) * d, flops=14 * d * pairs)
    qs, kvs = _lengths(c)
    T = sum(qs)
    if c["kind"] == "append":
        return dict(bytes=2 * 2 * 2 * T * Hkv * d, flops=0)
    W, ns = c["window"], c["sinks"]
    seen = 0                           # cached tokens that at least one new token sees
    for q, kv in zip(qs, kvs):
        if q:
            lo = max(0, kv - q - W + 1) if W else 0
            seen += kv - lo + min(ns, lo)
    return dict(bytes=2 * 2 * T * H * d + 2 * 2 * seen * Hkv * d, flops=4 * d * _pairs(c) * H)


# --- inputs -----------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    H, Hkv, d = c["H"], c["Hkv"], c["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    st = dict(case=c)
    if c["kind"] in ("fwd", "train"):
        B, L = c["B"], c["L"]
        st.update(q=normal(B, L, H, d), k=normal(B, L, Hkv, d), v=normal(B, L, Hkv, d))
        if c["kind"] == "train":
            st["dout"] = normal(B, L, H, d)
        return st
    qs, kvs = _lengths(c)
    page = c["page"]
    need = [-(-kv // page) for kv in kvs]
    n_pages = sum(need) + 3
    # pages are handed out in no order, as a cache does after some requests have come and gone
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    width = max(need)
    first = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    at = first[:, None] + torch.arange(width, device="cuda")[None]
    used = torch.arange(width, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(used, order[at.clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    cu = torch.tensor([0] + qs, device="cuda").cumsum(0).to(torch.int32)
    st.update(table=table, cu_q=cu, kv_len=torch.tensor(kvs, device="cuda", dtype=torch.int32),
              k_cache=normal(n_pages, page, Hkv, d), v_cache=normal(n_pages, page, Hkv, d))
    T = sum(qs)
    if c["kind"] == "append":
        st.update(k_new=normal(T, Hkv, d), v_new=normal(T, Hkv, d))
    else:
        st.update(q=normal(T, H, d))
    return st


# --- the plain form ---------------------------------------------------------------------
def _softmax_parts(q, k, qpos, kpos, kok, c):
    """q [N, M, H, d], k [N, S, Hkv, d] fp32; qpos [N, M], kpos and kok [N, S].
    Returns p [N, Hkv, G, M, S], normalised, and lse [N, Hkv, G, M]."""
    N, M, H, d = q.shape
    Hkv, W, ns = k.shape[2], c["window"], c["sinks"]
    qh = q.view(N, M, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4)
    s = torch.matmul(qh, k.permute(0, 2, 3, 1)[:, :, None]) * (1.0 / math.sqrt(d))
    see = (kpos[:, None, :] <= qpos[:, :, None]) & kok[:, None, :]
    if W:
        see &= (kpos[:, None, :] > qpos[:, :, None] - W) | (kpos[:, None, :] < ns)
    s = s.masked_fill(~see[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return p / total.clamp(min=1e-37), lse


def _heads_last(x):
    """[N, Hkv, G, M, d] -> [N, M, H, d]"""
    N, Hkv, G, M, d = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(N, M, Hkv * G, d)


def _blocks(c, dev):
    """Query positions [nb, BLOCK] and the key positions [nb, S] that a block can see."""
    L, W, ns = c["L"], c["window"], c["sinks"]
    nb = -(-L // _BLOCK)
    qpos = torch.arange(nb * _BLOCK, device=dev).view(nb, _BLOCK)
    win = torch.arange(-(W - 1), _BLOCK, device=dev)[None] + qpos[:, :1]
    sink = torch.arange(ns, device=dev)[None].expand(nb, ns)
    kpos = torch.cat([sink, win], 1)
    kok = torch.cat([sink < L, (win >= ns) & (win < L)], 1)
    return nb, qpos, kpos, kok


def _plain_sequence(st):
    c = st["case"]
    B, L, H, Hkv, d = c["B"], c["L"], c["H"], c["Hkv"], c["d"]
    dev = st["q"].device
    nb, qpos, kpos, kok = _blocks(c, dev)
    kat = kpos.clamp(0, L - 1)
    pad = nb * _BLOCK - L

    def queries(x):
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, pad))
        return x.view(B * nb, _BLOCK, x.shape[2], d)

    def back(x):
        return x.reshape(B, nb * _BLOCK, *x.shape[2:])[:, :L]

    q = queries(st["q"])
    k = st["k"].float()[:, kat].view(B * nb, -1, Hkv, d)
    v = st["v"].float()[:, kat].view(B * nb, -1, Hkv, d)
    p, lse = _softmax_parts(q, k, qpos.repeat(B, 1), kpos.repeat(B, 1), kok.repeat(B, 1), c)
    vh = v.permute(0, 2, 1, 3)[:, :, None]
    o32 = torch.matmul(p, vh)
    o = back(_heads_last(o32)).to(torch.bfloat16)
    lse = back(lse.permute(0, 3, 1, 2).reshape(B * nb, _BLOCK, H)).contiguous()
    if c["kind"] == "fwd":
        return [o.contiguous(), lse]
    G = H // Hkv
    g = queries(st["dout"]).view(B * nb, _BLOCK, Hkv, G, d).permute(0, 2, 3, 1, 4)
    dv = torch.matmul(p.transpose(-1, -2), g).sum(2)
    dp = torch.matmul(g, vh.transpose(-1, -2))
    delta = (g * o32).sum(-1, keepdim=True)
    ds = p * (dp - delta) * (1.0 / math.sqrt(d))
    dq = back(_heads_last(torch.matmul(ds, k.permute(0, 2, 1, 3)[:, :, None])))
    qh = q.view(B * nb, _BLOCK, Hkv, G, d).permute(0, 2, 3, 1, 4)
    dk = torch.matmul(ds.transpose(-1, -2), qh).sum(2)
    at = (kat[None] + L * torch.arange(B, device=dev)[:, None, None]).reshape(-1)
    keep = kok.repeat(B, 1).reshape(-1, 1, 1)

    def scatter(x):                    # [B nb, Hkv, S, d] onto the keys' places
        x = x.permute(0, 2, 1, 3).reshape(-1, Hkv, d)
        y = torch.zeros(B * L, Hkv, d, device=dev)
        return y.index_add_(0, at, torch.where(keep, x, 0.0)).view(B, L, Hkv, d)

    return [o.contiguous(), lse, dq.to(torch.bfloat16).contiguous(), scatter(dk).to(torch.bfloat16),
            scatter(dv).to(torch.bfloat16)]


def _plain_append(st):
    cu, kv, page = st["cu_q"].long(), st["kv_len"].long(), st["case"]["page"]
    T = st["k_new"].shape[0]
    tok = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    pos = kv[b] - cu[b + 1] + tok
    pg = st["table"].long()[b, pos // page]
    st["k_cache"][pg, pos % page] = st["k_new"]
    st["v_cache"][pg, pos % page] = st["v_new"]
    return [st["k_cache"], st["v_cache"]]


def _plain_paged(st):
    c = st["case"]
    H, Hkv, d, page, W, ns, M = (c[n] for n in ("H", "Hkv", "d", "page", "window", "sinks", "q_max"))
    cu, kv = st["cu_q"].long(), st["kv_len"].long()
    dev, T = cu.device, st["q"].shape[0]
    qlen = cu[1:] - cu[:-1]
    row = torch.arange(M, device=dev)[None]
    live = row < qlen[:, None]
    at = torch.where(live, cu[:-1, None] + row, T)
    q = torch.nn.functional.pad(st["q"].float(), (0, 0, 0, 0, 0, 1))[at]
    qpos = torch.where(live, kv[:, None] - qlen[:, None] + row, -1)
    cap = st["table"].shape[1] * page
    if W and ns + W + M - 1 < cap:
        win = (kv - qlen)[:, None] - W + 1 + torch.arange(W + M - 1, device=dev)[None]
        sink = torch.arange(ns, device=dev)[None].expand(len(kv), ns)
        kpos = torch.cat([sink, win], 1)
        kok = torch.cat([sink < kv[:, None], (win >= ns) & (win < kv[:, None])], 1)
    else:
        kpos = torch.arange(cap, device=dev)[None].expand(len(kv), cap)
        kok = kpos < kv[:, None]
    safe = torch.where(kok, kpos, 0)
    pg = st["table"].long().gather(1, safe // page).clamp(min=0)
    k = st["k_cache"][pg, safe % page].float()
    v = st["v_cache"][pg, safe % page].float()
    p, _ = _softmax_parts(q, k, qpos, kpos, kok, c)
    o = _heads_last(torch.matmul(p, v.permute(0, 2, 1, 3)[:, :, None]))
    out = torch.zeros(T + 1, H, d, device=dev, dtype=torch.bfloat16)
    out[at] = o.to(torch.bfloat16)
    return [out[:T]]


def run(state):
    st = state
    c = st["case"]
    if own:
        from retrieval_sparse_attention_gb300 import api
        if c["kind"] in ("fwd", "train"):
            o, lse = api.swa_sink_fwd(st["q"], st["k"], st["v"], window=c["window"], sinks=c["sinks"])
            if c["kind"] == "fwd":
                return [o, lse]
            dq, dk, dv = api.swa_sink_bwd(st["q"], st["k"], st["v"], o, lse, st["dout"], window=c["window"],
                                          sinks=c["sinks"])
            return [o, lse, dq, dk, dv]
        if c["kind"] == "append":
            api.paged_append(st["k_new"], st["v_new"], st["k_cache"], st["v_cache"], st["table"], st["cu_q"],
                             st["kv_len"])
            return [st["k_cache"], st["v_cache"]]
        o, _ = api.paged_attn(st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu_q"], st["kv_len"],
                              max_q=c["q_max"], window=c["window"], sinks=c["sinks"])
        return [o]
    if c["kind"] in ("fwd", "train"):
        return _plain_sequence(st)
    return _plain_append(st) if c["kind"] == "append" else _plain_paged(st)


# --- the definition in 64 bits ----------------------------------------------------------
def _exact_rows(q, k, v, first, kfirst, W, ns):
    """q [M, H, d] at positions first .., k and v [S, Hkv, d] at the positions in kfirst [S]; 64 bits.
    Returns weights [H, M, S] and lse [H, M], with key heads repeated for their query heads."""
    G = q.shape[1] // k.shape[1]
    kk = k.repeat_interleave(G, 1)
    s = torch.einsum("mhd,shd->hms", q, kk) / math.sqrt(q.shape[2])
    qp = torch.arange(first, first + q.shape[0], device=q.device)[:, None]
    hidden = kfirst[None] > qp
    if W:
        hidden = hidden | ((kfirst[None] <= qp - W) & (kfirst[None] >= ns))
    s = s.masked_fill(hidden[None], float("-inf"))
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[..., None]), lse, kk, v.repeat_interleave(G, 1)


def _exact_keys(lo_row, hi_row, W, ns, dev):
    """Positions that rows lo_row .. hi_row - 1 can see between them."""
    lo = max(0, lo_row - W + 1) if W else 0
    return torch.cat([torch.arange(min(ns, lo), device=dev), torch.arange(lo, hi_row, device=dev)])


def exact(case, seed):
    c = case
    if c["kind"] == "append":
        return None
    st = prepare(case, seed)
    W, ns, H, Hkv, d = c["window"], c["sinks"], c["H"], c["Hkv"], c["d"]
    dev = st["q"].device
    if c["kind"] == "paged":
        qs, kvs = _lengths(c)
        q, out, row = st["q"].double(), [], 0
        for b, (n, kv) in enumerate(zip(qs, kvs)):
            for t0 in range(0, n, 256):
                t1 = min(n, t0 + 256)
                pos = _exact_keys(kv - n + t0, kv - n + t1, W, ns, dev)
                pg = st["table"][b][pos // c["page"]].long()
                k, v = (st[x][pg, pos % c["page"]].double() for x in ("k_cache", "v_cache"))
                w, _, _, vv = _exact_rows(q[row + t0:row + t1], k, v, kv - n + t0, pos, W, ns)
                out.append(torch.einsum("hms,shd->mhd", w, vv))
            row += n
        return [torch.cat(out) if out else q.new_zeros(0, H, d)]
    B, L, train = c["B"], c["L"], c["kind"] == "train"
    o = torch.empty(B, L, H, d, device=dev, dtype=torch.float64)
    lse = torch.empty(B, L, H, device=dev, dtype=torch.float64)
    if train:
        dq = torch.empty_like(o)
        dk = torch.zeros(B, L, Hkv, d, device=dev, dtype=torch.float64)
        dv = torch.zeros_like(dk)
    step = max(128, min(2048, W))
    for b in range(B):
        for t0 in range(0, L, step):
            t1 = min(L, t0 + step)
            pos = _exact_keys(t0, t1, W, ns, dev)
            q, k, v = st["q"][b, t0:t1].double(), st["k"][b, pos].double(), st["v"][b, pos].double()
            w, ls, kk, vv = _exact_rows(q, k, v, t0, pos, W, ns)
            o[b, t0:t1] = torch.einsum("hms,shd->mhd", w, vv)
            lse[b, t0:t1] = ls.transpose(0, 1)
            if train:
                g = st["dout"][b, t0:t1].double()
                dw = torch.einsum("mhd,shd->hms", g, vv)
                dz = w * (dw - (w * dw).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[b, t0:t1] = torch.einsum("hms,shd->mhd", dz, kk)
                fold = lambda x: x.view(len(pos), Hkv, H // Hkv, d).sum(2)  # noqa: E731
                dk[b].index_add_(0, pos, fold(torch.einsum("hms,mhd->shd", dz, q)))
                dv[b].index_add_(0, pos, fold(torch.einsum("hms,mhd->shd", w, g)))
    return [o, lse, dq, dk, dv] if train else [o, lse]
