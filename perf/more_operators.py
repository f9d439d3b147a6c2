"""Timed cases of rotary positions, of the pages of a paged K/V cache, and of window attention with transformed scores.

Six operators: rotary positions of queries and keys (with their gradient); a
serving step's reservation of pages and its rotated write into the cache; the
fork of sequences that share pages; the compaction of a cache; the attention
over a window with sinks whose scores are capped by a tanh or biased by the
distance, with its gradients, and the same over the paged cache.

``run`` computes an operator in plain 32-bit torch operations, or, where
``own`` is true, by the calls a user makes of this package.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_BLOCK = 256          # queries that the plain form of the attention takes together


# --- cases ------------------------------------------------------------------------------
def listed():
    return [
        # one short prompt: the time of the launch counts
        dict(name="rope_b1_517", kind="rope", B=1, L=517, H=12, Hkv=12, d=64, rot=64, inter=False, scaling="none", start=0),
        # a training step's rotation and its gradient, at the batch of the 12-head model
        dict(name="rope_b8_16k", kind="rope", B=8, L=16384, H=12, Hkv=12, d=64, rot=64, inter=False, scaling="none", start=0),
        # a generated token of each of 64 requests, behind a window whose pages are let go: latency
        dict(name="step_b64_tokens", kind="step", B=64, q_max=1, q_min=1, kv_max=2048, kv_min=64, ragged=11, H=24, Hkv=8,
             d=128, rot=64, inter=True, page=16, window=512, sinks=4),
        # eight prompt chunks of uneven length
        dict(name="step_b8_chunks", kind="step", B=8, q_max=2048, q_min=900, kv_max=4096, kv_min=500, ragged=12, H=12,
             Hkv=12, d=64, rot=64, inter=False, page=64, window=0, sinks=0),
        # two requests with four beams each, which change places
        dict(name="fork_b8_beams", kind="fork", B=8, group=4, kv_max=777, kv_min=300, ragged=13, Hkv=12, d=64, page=16),
        # 64 requests with four beams each, wide pages
        dict(name="fork_b256_beams", kind="fork", B=256, group=4, kv_max=6000, kv_min=1000, ragged=14, Hkv=8, d=128,
             page=128),
        # a small cache that some requests have left
        dict(name="compact_100_pages", kind="compact", n_pages=100, used=41, B=5, moves=50, Hkv=12, d=64, page=16),
        # half of a large cache: bound by the bytes that move
        dict(name="compact_8k_pages", kind="compact", n_pages=8192, used=4100, B=64, moves=2100, Hkv=8, d=128, page=64),
        # a training step on short odd sequences, distance bias, three query heads to a key head
        dict(name="train_b3_1000_bias", kind="train", B=3, L=1000, H=6, Hkv=2, d=64, window=200, sinks=1, cap=0.0, bias=True),
        # a training step of the 12-head model at its own batch, capped scores
        dict(name="train_b8_16k_cap", kind="train", B=8, L=16384, H=12, Hkv=12, d=64, window=512, sinks=4, cap=20.0,
             bias=False),
        # one token of each of 32 long requests over their whole caches, capped scores: bound by the cache's bytes
        dict(name="paged_b32_tokens_32k_cap", kind="paged", B=32, q_max=1, q_min=1, kv_max=32768, kv_min=4096, ragged=15,
             H=24, Hkv=8, d=128, page=64, window=0, sinks=0, cap=30.0, bias=False),
        # a serving batch: idle slots, single tokens and prompt chunks together, distance bias within the window
        dict(name="paged_b48_mixed_bias", kind="paged", B=48, q_max=512, q_min=0, kv_max=6000, kv_min=512, ragged=16,
             H=12, Hkv=12, d=64, page=16, window=512, sinks=4, cap=0.0, bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rope", "step", "fork", "compact", "train", "train", "paged", "paged"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 12])
    H = Hkv * rng.choice([1, 2, 3, 4, 8] if Hkv <= 4 else [1, 2, 3])
    page = rng.choice([16, 32, 64, 128])
    inter = rng.choice([False, True])
    ragged = rng.randrange(1 << 20)
    if kind == "rope":
        B, L = _log_int(rng, 1, 8), _log_int(rng, 1, 32768)
        d = rng.choice([32, 64, 128])
        while B * L * (H + Hkv) * d > 1.9e8:
            L = max(1, L // 2 + rng.randrange(3))
        return dict(kind=kind, B=B, L=L, H=H, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2]), inter=inter,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), start=rng.choice([0, 0, _log_int(rng, 1, 1000000)]))
    if kind == "step":
        B = _log_int(rng, 1, 128)
        q_max = rng.choice([1, 1, _log_int(rng, 2, 2048)])
        kv_max = _log_int(rng, 16, 8192)
        while B * q_max * (H + 2 * Hkv) * d > 4e7 or B * (kv_max + q_max) * Hkv * d > 2e8:
            q_max = max(1, q_max * 2 // 3)
            kv_max = max(16, kv_max * 2 // 3 + rng.randrange(3))
            B = max(1, B * 5 // 6)
        return dict(kind=kind, B=B, q_max=q_max, q_min=1 if q_max == 1 else rng.choice([0, 1, q_max]), kv_max=kv_max,
                    kv_min=rng.choice([0, kv_max // 4, kv_max]), ragged=ragged, H=H, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d // 2]), inter=inter, page=page,
                    **rng.choice([dict(window=0, sinks=0), dict(window=_log_int(rng, 16, 2048), sinks=rng.choice([0, 1, 4, 33]))]))
    if kind == "fork":
        group = rng.choice([2, 3, 4, 8])
        B, kv_max = group * _log_int(rng, 1, 48), _log_int(rng, 32, 6000)
        while B * (kv_max + page) * Hkv * d > 5e8:
            kv_max = max(32, kv_max * 2 // 3)
            B = max(group, B // 2 // group * group)
        return dict(kind=kind, B=B, group=group, kv_max=kv_max, kv_min=rng.choice([1, kv_max // 3, kv_max]), ragged=ragged,
                    Hkv=Hkv, d=d, page=page)
    if kind == "compact":
        n_pages = _log_int(rng, 40, 20000)
        while n_pages * page * Hkv * d > 5e8:
            n_pages = max(40, n_pages // 2)
        used = rng.randrange(n_pages // 8, n_pages - n_pages // 16)
        return dict(kind=kind, n_pages=n_pages, used=used, B=rng.randint(1, 40), Hkv=Hkv, d=d, page=page,
                    moves=rng.choice([n_pages // 2, max(1, n_pages // 10)]))
    score = rng.choice([dict(cap=rng.choice([5.0, 20.0, 50.0]), bias=False), dict(cap=0.0, bias=True)])
    sinks = rng.choice([0, 1, 4, 16, 33, 64])
    if kind == "train":
        # (16 tokens at least: the first one's query gradient is zero whatever the inputs)
        B, L, W = _log_int(rng, 1, 8), _log_int(rng, 16, 32768), _log_int(rng, 16, 2048)
        while B * L * H * d * (W + sinks + 128) > 2.5e10:      # under half the largest listed one
            L = max(16, L // 2 + rng.randrange(3))
            B = max(1, B - 1)
        return dict(kind=kind, B=B, L=L, H=H, Hkv=Hkv, d=d, window=W, sinks=sinks, **score)
    B = _log_int(rng, 1, 64)
    q_max = rng.choice([1, 1, _log_int(rng, 2, 2048)])
    kv_max = max(q_max, _log_int(rng, 16, 32768))
    while B * q_max * kv_max * H * d > 6e10 or B * kv_max * Hkv * d > 5e8:
        kv_max = max(16, kv_max // 2 + rng.randrange(5))
        q_max = min(q_max, kv_max)
        B = max(1, B * 3 // 4)
    window = rng.choice([0, _log_int(rng, 16, 4096)])
    kv_min = max(q_max, kv_max // rng.choice([1, 4, 20]))
    return dict(kind=kind, B=B, q_max=q_max, q_min=1 if q_max == 1 else rng.choice([0, 1, q_max]), kv_max=max(kv_max, kv_min),
                kv_min=kv_min, ragged=ragged, H=H, Hkv=Hkv, d=d, page=page, window=window, sinks=sinks if window else 0, **score)


def _lengths(c):
    """New tokens and earlier tokens of each sequence of a case with a cache."""
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
        kv = c["kv_max"] if i == 0 else r.randint(c["kv_min"], c["kv_max"])
        qs.append(n)
        kvs.append(kv if c["kind"] == "step" else max(0, kv - n))
    return qs, kvs


def _beams(c):
    """Shared prompt pages, tokens and parents of the slots of a fork."""
    r = random.Random(c["ragged"])
    G, page = c["group"], c["page"]
    shared, lens, parents = [], [], []
    for g in range(c["B"] // G):
        n = c["kv_max"] if g == 0 else r.randint(c["kv_min"], c["kv_max"])
        s = r.randint(0, n) // page
        gone = r.random() < 0.1                          # a request that has ended
        for i in range(G):
            shared.append(s)
            lens.append(n)
            # beams go on from any beam of their request; some end
            parents.append(-1 if gone or r.random() < 0.05 else g * G + r.randrange(G))
    return shared, lens, parents


def _pairs(c):
    """(query, visible key) pairs of one query head."""
    W, ns = c["window"], c["sinks"]
    if c["kind"] == "train":
        spans = [(0, c["L"])] * c["B"]
    else:
        spans = [(kv, kv + q) for q, kv in zip(*_lengths(c))]

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
    d, Hkv = c["d"], c["Hkv"]
    if c["kind"] == "rope":
        n = c["B"] * c["L"] * (c["H"] + Hkv)
        return dict(bytes=2 * 2 * 2 * n * d, flops=2 * 3 * n * c["rot"])
    if c["kind"] == "step":
        T = sum(_lengths(c)[0])
        return dict(bytes=2 * 2 * T * (c["H"] + 2 * Hkv) * d + 4 * 4 * c["B"], flops=3 * T * (c["H"] + Hkv) * c["rot"])
    if c["kind"] == "fork":
        _, lens, parents = _beams(c)
        entries = sum(-(-lens[p] // c["page"]) for p in parents if p >= 0)
        taken, copies = set(), 0
        for p in parents:
            copies += p >= 0 and p in taken and lens[p] % c["page"] > 0
            taken.add(p)
        return dict(bytes=4 * (2 * entries + 3 * c["B"]) + copies * 2 * 2 * 2 * c["page"] * Hkv * d, flops=0)
    if c["kind"] == "compact":
        # (of the pages above the mark, those in use: a share of `used` by chance)
        moved = min(c["moves"], round(c["used"] * (c["n_pages"] - c["used"]) / c["n_pages"]))
        return dict(bytes=moved * 2 * 2 * 2 * c["page"] * Hkv * d + 4 * (2 * c["used"] + c["n_pages"] // 32), flops=0)
    H = c["H"]
    if c["kind"] == "train":
        tok = c["B"] * c["L"]
        byt = 2 * 2 * tok * (2 * H + 2 * Hkv) * d + 4 * tok * H
        return dict(bytes=byt, flops=14 * d * _pairs(c) * H)
    qs, kvs = _lengths(c)
    W, ns = c["window"], c["sinks"]
    seen = 0                           # cached tokens that at least one new token sees
    for q, kv in zip(qs, kvs):
        if q:
            lo = max(0, kv - W + 1) if W else 0
            seen += kv + q - lo + min(ns, lo)
    return dict(bytes=2 * 2 * sum(qs) * H * d + 2 * 2 * seen * Hkv * d, flops=4 * d * _pairs(c) * H)


# --- inputs -----------------------------------------------------------------------------
def _inv_freq(c, dev):
    """Angle of a pair a position, 64 bits: plain, or scaled for contexts eight times as long."""
    rot = c["rot"]
    i = torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot
    scaling, factor = c.get("scaling", "none"), 8.0
    base = 10000.0 * (factor ** (rot / (rot - 2)) if scaling == "ntk" else 1.0)
    inv = base ** -i
    if scaling == "linear":
        inv = inv / factor
    if scaling == "yarn":              # pairs that turn often over the 4096 trained tokens stay, slow ones are stretched
        turns = 4096 * inv / (2 * math.pi)
        keep = ((torch.log(turns) - 0.0) / math.log(32.0)).clamp(0, 1)
        inv = inv * keep + inv / factor * (1 - keep)
    return inv


def _table_of(inv):
    """A pair's angle as a 64-bit fraction of a turn."""
    turns = inv / (2 * math.pi)
    return ((turns - turns.round()) * 2.0 ** 64).to(torch.int64)


def _words(refs):
    """The free pages as bits, 32 a word."""
    n = refs.numel()
    free = torch.nn.functional.pad(refs == 0, (0, -n % 32)).view(-1, 32).long()
    w = (free << torch.arange(32, device=refs.device)).sum(1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _ints(st, **parts):
    """The allocator's integers as parts of one tensor, with a snapshot that a pass begins from: a step
    that is tried again goes back to it."""
    live = torch.cat([x.reshape(-1) for x in parts.values()])
    st["live"], st["snapshot"], at = live, live.clone(), 0
    for name, x in parts.items():
        st[name] = live[at:at + x.numel()].view(x.shape)
        at += x.numel()


def _pool(refs):
    """Counts, free bits, and as many scratch words as pages."""
    return torch.cat([refs, _words(refs), torch.zeros_like(refs)])


def _pad4(x):
    """Whole 16-byte units, so that the next part of one tensor is aligned."""
    return torch.nn.functional.pad(x, (0, -x.numel() % 4))


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    Hkv, d = c["Hkv"], c["d"]
    i32 = torch.int32

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * scale).to(torch.bfloat16)

    st = dict(case=c)
    if c["kind"] == "rope":
        B, L, H = c["B"], c["L"], c["H"]
        st.update(q=normal(B, L, H, d), k=normal(B, L, Hkv, d), dq=normal(B, L, H, d), dk=normal(B, L, Hkv, d),
                  inv=_inv_freq(c, dev))
        st["freqs"] = _table_of(st["inv"])
        return st
    if c["kind"] == "train" or c["kind"] == "paged":
        H = c["H"]
        st["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H) if c["bias"] else None
    if c["kind"] == "train":
        B, L = c["B"], c["L"]
        # (scores of a few units, some of them near the cap)
        st.update(q=normal(B, L, H, d, scale=3.0), k=normal(B, L, Hkv, d), v=normal(B, L, Hkv, d), dout=normal(B, L, H, d))
        return st
    page = c["page"]
    if c["kind"] == "compact":
        n, used, B = c["n_pages"], c["used"], c["B"]
        order = torch.randperm(n, generator=g, device=dev)
        width = -(-used // B)
        table = torch.full((B * width,), -1, device=dev, dtype=i32)
        table[:used] = order[:used].to(i32)
        refs = torch.zeros(n, device=dev, dtype=i32)
        refs[order[:used]] = 1
        _ints(st, pool=_pad4(_pool(refs)), table=table.view(B, width))
        st["pool"] = st["pool"][:2 * n + -(-n // 32)]
        st.update(k_cache=normal(n, page, Hkv, d), v_cache=normal(n, page, Hkv, d))
        return st
    if c["kind"] == "fork":
        shared, lens, parents = (torch.tensor(x, device=dev) for x in _beams(c))
        B, G = c["B"], c["group"]
        need = -(-lens // page)
        width = int(need.max())
        col = torch.arange(width, device=dev)[None]
        lead = torch.arange(B, device=dev)[:, None] // G * G          # the slot whose pages a request's beams share
        at = torch.where(col < shared[:, None], lead, torch.arange(B, device=dev)[:, None]) * width + col
        has = col < need[:, None]
        first = torch.zeros(B * width, device=dev, dtype=torch.long).index_fill_(0, at[has], 1)
        number = first.cumsum(0) - 1
        n = int(first.sum()) + B
        order = torch.randperm(n, generator=g, device=dev)
        table = torch.where(has, order[number[at].clamp(min=0)], -1).to(i32)
        refs = torch.zeros(n, device=dev, dtype=i32)
        refs.index_add_(0, table[has].long(), torch.ones_like(table[has]))
        _ints(st, pool=_pad4(_pool(refs)), kv_len=_pad4(lens.to(i32)), table=table)
        st.update(pool=st["pool"][:2 * n + -(-n // 32)], kv_len=st["kv_len"][:B], parent=parents.to(i32),
                  k_cache=normal(n, page, Hkv, d), v_cache=normal(n, page, Hkv, d))
        return st
    qs, kvs = _lengths(c)
    H, B = c["H"], c["B"]
    step = c["kind"] == "step"
    q, kv = torch.tensor(qs, device=dev), torch.tensor(kvs, device=dev)
    have = -(-(kv if step else kv + q) // page)
    width = max(1, int((-(-(kv + q) // page)).max()))
    col = torch.arange(width, device=dev)[None]
    has = col < have[:, None]
    if step and c["window"]:           # what left the window has been let go, up to a step ago
        gone = ((kv - 1 - c["window"] + 1).clamp(min=0) // page)[:, None]
        has &= (col >= gone) | (col < -(-c["sinks"] // page))
    n = int(has.sum()) + int((-(-(kv + q) // page) - have).sum()) + 3
    # pages are handed out in no order, as a cache does after some requests have come and gone
    order = torch.randperm(n, generator=g, device=dev)
    number = (has.reshape(-1).cumsum(0) - 1).view(B, width)
    table = torch.where(has, order[number.clamp(min=0)], -1).to(i32)
    cu = torch.cat([q.new_zeros(1), q.cumsum(0)]).to(i32)
    st.update(cu_q=cu, k_cache=normal(n, page, Hkv, d), v_cache=normal(n, page, Hkv, d))
    T = sum(qs)
    if step:
        refs = torch.zeros(n, device=dev, dtype=i32)
        refs[table[has].long()] = 1
        _ints(st, pool=_pad4(_pool(refs)), kv_len=_pad4(kv.to(i32)), table=table)
        st.update(pool=st["pool"][:2 * n + -(-n // 32)], kv_len=st["kv_len"][:B], q=normal(T, H, d), k_new=normal(T, Hkv, d),
                  v_new=normal(T, Hkv, d), inv=_inv_freq(c, dev))
        st["freqs"] = _table_of(st["inv"])
        return st
    st.update(table=table.contiguous(), kv_len=(kv + q).to(i32), q=normal(T, H, d, scale=3.0))
    return st


# --- the plain forms: rotary positions ---------------------------------------------------
def _rotate(x, pos, inv, inter, sign=1.0):
    """x [..., T, H, d] at positions [..., T]: its first 2 len(inv) columns turned, in 32 bits."""
    rot = 2 * inv.numel()
    a = pos.double()[..., None] * inv
    a = a - (2 * math.pi) * torch.round(a / (2 * math.pi))
    cos, sin = torch.cos(a).float()[..., None, :], sign * torch.sin(a).float()[..., None, :]
    y = x.float()
    if inter:
        u, w = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([u * cos - w * sin, u * sin + w * cos], -1).flatten(-2)
    else:
        u, w = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([u * cos - w * sin, u * sin + w * cos], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_rope(st):
    c = st["case"]
    pos = (c["start"] + torch.arange(c["L"], device=st["q"].device))[None].expand(c["B"], c["L"])
    turn = lambda x, s: _rotate(x, pos, st["inv"], c["inter"], s)  # noqa: E731
    return [turn(st["q"], 1.0), turn(st["k"], 1.0), turn(st["dq"], -1.0), turn(st["dk"], -1.0)]


# --- the plain forms: pages --------------------------------------------------------------
def _state(pool, n):
    return pool[:n + -(-n // 32)]


def _free_list(refs):
    """Free pages in ascending order, then anything; how many."""
    free = refs == 0
    rank = free.long().cumsum(0) - 1
    out = torch.zeros(refs.numel() + 1, device=refs.device, dtype=torch.long)
    out.scatter_(0, torch.where(free, rank, refs.numel()), torch.arange(refs.numel(), device=refs.device))
    return out, free.sum()


def _plain_reserve(st):
    c = st["case"]
    table, kv, cu, page = st["table"], st["kv_len"], st["cu_q"].long(), c["page"]
    n = st["k_cache"].shape[0]
    refs, width = st["pool"][:n], table.shape[1]
    new, old = cu[1:] - cu[:-1], kv.long()
    col = torch.arange(width, device=table.device)[None]
    if c["window"]:
        lo, hi = -(-c["sinks"] // page), (old - c["window"] + 1).clamp(min=0) // page
        inside = (col >= lo) & (col < hi[:, None]) & (new > 0)[:, None]
        held = inside & (table >= 0)
        # downwards from the window, as far as entries hold pages
        run = torch.where(inside, held, True).flip(1).long().cumprod(1).flip(1) > 0
        let = held & run
        refs.index_add_(0, torch.where(let, table, 0).reshape(-1).long(), -let.reshape(-1).to(torch.int32))
        table.copy_(torch.where(let, -1, table))
    lack = (table < 0) & (col >= (old // page)[:, None]) & (col < (-(-(old + new) // page))[:, None]) & (new > 0)[:, None]
    need = lack.sum(1)
    end = need.cumsum(0)
    free, count = _free_list(refs)
    fits = (old + new <= width * page) & ((end <= count) | (need == 0))
    rank = (end - need)[:, None] + lack.long().cumsum(1) - 1
    got = lack & fits[:, None]
    pages = free[torch.where(got, rank, 0)]
    table.copy_(torch.where(got, pages.to(torch.int32), table))
    refs.index_add_(0, torch.where(got, pages, 0).reshape(-1), got.reshape(-1).to(torch.int32))
    kv.copy_(torch.where(fits, old + new, -1 - old))
    st["pool"][n:n + -(-n // 32)] = _words(refs)


def _plain_step(st):
    c = st["case"]
    st["live"].copy_(st["snapshot"])
    _plain_reserve(st)
    cu, kv, page = st["cu_q"].long(), st["kv_len"].long(), c["page"]
    tok = torch.arange(st["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    pos = kv[b] - cu[b + 1] + tok
    pg = st["table"].long()[b, pos // page]
    st["k_cache"][pg, pos % page] = _rotate(st["k_new"], pos, st["inv"], c["inter"])
    st["v_cache"][pg, pos % page] = st["v_new"]
    q = _rotate(st["q"], pos, st["inv"], c["inter"])
    return [q, st["k_cache"], st["v_cache"], st["table"], st["kv_len"], _state(st["pool"], st["k_cache"].shape[0])]


def _plain_copy(st, pairs):
    src, dst = pairs[:, 0].long(), pairs[:, 1].long()
    move = dst >= 0
    # (entries without a move repeat one that is; where there is none, page 0 is written onto itself)
    some = move.long().argmax()
    src, dst = (torch.where(move, x, x[some].clamp(min=0)) for x in (src, dst))
    for x in (st["k_cache"], st["v_cache"]):
        x[dst] = x[src]


def _plain_fork(st):
    c = st["case"]
    st["live"].copy_(st["snapshot"])
    table, kv, page, parent = st["table"], st["kv_len"], c["page"], st["parent"].long()
    B, width = table.shape
    n = st["k_cache"].shape[0]
    refs, dev = st["pool"][:n], table.device
    old, lens = table.clone(), kv.long()
    slot = torch.arange(B, device=dev)
    live = parent >= 0
    src = parent.clamp(min=0)
    # of a slot's children it goes on itself, or else the first of them keeps its last page
    lowest = torch.full((B,), B, device=dev).scatter_reduce_(0, src, torch.where(live, slot, B), "amin")
    keeper = torch.where(parent == slot, slot, lowest)
    part, last = lens % page > 0, (lens // page).clamp(max=width - 1)
    held = old.gather(1, last[:, None])[:, 0]
    copy = live & (keeper[src] != slot) & part[src] & (held[src] >= 0)
    free, _ = _free_list(refs)                           # (as many as slots, at least)
    fresh = free[torch.where(copy, copy.long().cumsum(0) - 1, 0)]
    pairs = torch.where(copy[:, None], torch.stack([held[src].long(), fresh], 1), -1).to(torch.int32)
    col = torch.arange(width, device=dev)[None]
    table.copy_(torch.where(live[:, None], torch.where(copy[:, None] & (col == last[src][:, None]), fresh[:, None].to(torch.int32), old[src]), -1))
    kv.copy_(torch.where(live, lens[src], 0))
    # counts: every entry of the rows that were goes, every entry of those that are comes
    one = lambda t: (t >= 0).reshape(-1).to(torch.int32)  # noqa: E731
    refs.index_add_(0, old.clamp(min=0).reshape(-1).long(), -one(old))
    refs.index_add_(0, table.clamp(min=0).reshape(-1).long(), one(table))
    st["pool"][n:n + -(-n // 32)] = _words(refs)
    _plain_copy(st, pairs)
    return [st["k_cache"], st["v_cache"], table, kv, pairs, _state(st["pool"], n)]


def _plain_compact(st):
    c = st["case"]
    st["live"].copy_(st["snapshot"])
    n, moves, table = c["n_pages"], c["moves"], st["table"]
    refs = st["pool"][:n]
    used = refs > 0
    page, total = torch.arange(n, device=refs.device), used.sum()
    hole, high = ~used & (page < total), used & (page >= total)
    m = hole.sum()
    rank = torch.where(hole, hole.long().cumsum(0) - 1, m - high.long().cumsum(0))
    do = (hole | high) & (rank < moves)
    pairs = torch.full((moves + 1, 2), -1, device=refs.device, dtype=torch.int32)
    pairs[torch.where(do & high, rank, moves), 0] = page.to(torch.int32)
    pairs[torch.where(do & hole, rank, moves), 1] = page.to(torch.int32)
    pairs = pairs[:moves]
    src, dst = (torch.where(pairs[:, i] >= 0, pairs[:, i].long(), n) for i in (0, 1))
    wide = torch.cat([refs, refs.new_zeros(1)])
    wide[dst] = wide[src]
    to = torch.arange(n + 1, device=refs.device)
    to[src] = dst
    wide[src] = 0
    refs.copy_(wide[:n])
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    st["pool"][n:n + -(-n // 32)] = _words(refs)
    _plain_copy(st, pairs)
    return [st["k_cache"], st["v_cache"], table, pairs, _state(st["pool"], n)]


# --- the plain forms: attention ----------------------------------------------------------
def _scores(q, k, qpos, kpos, kok, c, slopes):
    """q [N, M, H, d], k [N, S, Hkv, d] fp32; qpos [N, M], kpos and kok [N, S].
    Returns p [N, Hkv, G, M, S], normalised, lse [N, Hkv, G, M] and the cap's slope, or None."""
    N, M, H, d = q.shape
    Hkv, W, ns = k.shape[2], c["window"], c["sinks"]
    qh = q.view(N, M, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4)
    s = torch.matmul(qh, k.permute(0, 2, 3, 1)[:, :, None]) * (1.0 / math.sqrt(d))
    bend = None
    if c["cap"]:
        t = torch.tanh(s / c["cap"])
        s, bend = t * c["cap"], 1 - t * t
    if slopes is not None:
        far = (qpos[:, :, None] - kpos[:, None, :]).float()
        s = s - slopes.view(1, Hkv, H // Hkv, 1, 1) * far[:, None, None]
    see = (kpos[:, None, :] <= qpos[:, :, None]) & kok[:, None, :]
    if W:
        see &= (kpos[:, None, :] > qpos[:, :, None] - W) | (kpos[:, None, :] < ns)
    s = s.masked_fill(~see[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return p / total.clamp(min=1e-37), lse, bend


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


def _plain_train(st):
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
    p, lse, bend = _scores(q, k, qpos.repeat(B, 1), kpos.repeat(B, 1), kok.repeat(B, 1), c, st["slopes"])
    vh = v.permute(0, 2, 1, 3)[:, :, None]
    o32 = torch.matmul(p, vh)
    o = back(_heads_last(o32)).to(torch.bfloat16)
    lse = back(lse.permute(0, 3, 1, 2).reshape(B * nb, _BLOCK, H)).contiguous()
    G = H // Hkv
    g = queries(st["dout"]).view(B * nb, _BLOCK, Hkv, G, d).permute(0, 2, 3, 1, 4)
    dv = torch.matmul(p.transpose(-1, -2), g).sum(2)
    dp = torch.matmul(g, vh.transpose(-1, -2))
    delta = (g * o32).sum(-1, keepdim=True)
    ds = p * (dp - delta) * (1.0 / math.sqrt(d))
    del dp, p
    if bend is not None:
        ds *= bend
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
    p, _, _ = _scores(q, k, qpos, kpos, kok, c, st["slopes"])
    o = _heads_last(torch.matmul(p, v.permute(0, 2, 1, 3)[:, :, None]))
    out = torch.zeros(T + 1, H, d, device=dev, dtype=torch.bfloat16)
    out[at] = o.to(torch.bfloat16)
    return [out[:T]]


# --- a pass ------------------------------------------------------------------------------
def _own(st):
    from retrieval_sparse_attention_gb300 import api
    c = st["case"]
    if c["kind"] == "rope":
        kw = dict(start=c["start"], interleaved=c["inter"])
        return [*api.rope(st["q"], st["k"], st["freqs"], **kw), *api.rope_bwd(st["dq"], st["dk"], st["freqs"], **kw)]
    if c["kind"] == "train":
        kw = dict(window=c["window"], sinks=c["sinks"], softcap=c["cap"], slopes=st["slopes"])
        o, lse = api.swa_sink_fwd(st["q"], st["k"], st["v"], **kw)
        return [o, lse, *api.swa_sink_bwd(st["q"], st["k"], st["v"], o, lse, st["dout"], **kw)]
    if c["kind"] == "paged":
        o, _ = api.paged_attn(st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu_q"], st["kv_len"], max_q=c["q_max"],
                              window=c["window"], sinks=c["sinks"], softcap=c["cap"], slopes=st["slopes"])
        return [o]
    st["live"].copy_(st["snapshot"])
    k, v, table, pool, page = st["k_cache"], st["v_cache"], st["table"], st["pool"], c["page"]
    state = _state(pool, k.shape[0])
    if c["kind"] == "step":
        api.paged_reserve(table, st["cu_q"], st["kv_len"], pool, page=page, window=c["window"], sinks=c["sinks"])
        q = api.paged_rope_append(st["q"], st["k_new"], st["v_new"], st["freqs"], k, v, table, st["cu_q"], st["kv_len"],
                                  interleaved=c["inter"])
        return [q, k, v, table, st["kv_len"], state]
    if c["kind"] == "fork":
        pairs = api.paged_fork(table, st["kv_len"], st["parent"], pool, page=page)
        api.paged_copy(k, v, pairs)
        return [k, v, table, st["kv_len"], pairs, state]
    pairs = api.paged_compact(table, pool, max_moves=c["moves"])
    api.paged_copy(k, v, pairs)
    return [k, v, table, pairs, state]


def run(state):
    if own:
        return _own(state)
    plain = dict(rope=_plain_rope, step=_plain_step, fork=_plain_fork, compact=_plain_compact, train=_plain_train,
                 paged=_plain_paged)
    return plain[state["case"]["kind"]](state)


# --- the definitions in 64 bits ----------------------------------------------------------
def _turned(x, pos, inv, inter, sign):
    """Pairs as complex numbers times e^(i angle)."""
    rot = 2 * inv.numel()
    w = torch.exp(1j * sign * torch.remainder(pos.double()[..., None] * inv, 2 * math.pi))[..., None, :]
    y = x.double().clone()
    if inter:
        first, second = slice(0, rot, 2), slice(1, rot, 2)
    else:
        first, second = slice(0, rot // 2), slice(rot // 2, rot)
    z = torch.complex(y[..., first], y[..., second]) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rows(q, k, v, first, kpos, c, slopes):
    """q [M, H, d] at positions first .., k and v [S, Hkv, d] at the positions kpos; 64 bits.
    Returns weights [H, M, S], lse [H, M], the scores' derivative by the products', and the
    keys and values repeated for their query heads."""
    H, d = q.shape[1:]
    G = H // k.shape[1]
    kk = k.repeat_interleave(G, 1)
    s = torch.einsum("mhd,shd->hms", q, kk) / math.sqrt(d)
    turn = 1.0 / math.sqrt(d)
    if c["cap"]:
        turn = turn / torch.cosh(s / c["cap"]) ** 2
        s = c["cap"] * torch.tanh(s / c["cap"])
    qp = torch.arange(first, first + q.shape[0], device=q.device)[:, None]
    if slopes is not None:
        s = s + slopes.double()[:, None, None] * (kpos[None] - qp).double()[None]
    hidden = kpos[None] > qp
    if c["window"]:
        hidden = hidden | ((kpos[None] <= qp - c["window"]) & (kpos[None] >= c["sinks"]))
    s = s.masked_fill(hidden[None], float("-inf"))
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[..., None]), lse, turn, kk, v.repeat_interleave(G, 1)


def _exact_keys(lo_row, hi_row, W, ns, dev):
    """Positions that rows lo_row .. hi_row - 1 can see between them."""
    lo = max(0, lo_row - W + 1) if W else 0
    return torch.cat([torch.arange(min(ns, lo), device=dev), torch.arange(lo, hi_row, device=dev)])


def _places(c, table, n, qs, kvs):
    """(page, row) of every new token of a step, one sequence after the other."""
    page, out = c["page"], []
    for row, q, kv in zip(table, qs, kvs):
        i = max(0, kv - c["window"] + 1) // page - 1 if c["window"] and q else -1
        while i >= -(-c["sinks"] // page) and row[i] >= 0:
            row[i] = -1
            i -= 1
    used = {x for row in table for x in row}
    free = (x for x in range(n) if x not in used)
    for row, q, kv in zip(table, qs, kvs):
        for p in range(kv, kv + q):
            if row[p // page] < 0:
                row[p // page] = next(free)
            out.append((row[p // page], p % page))
    return out


def exact(case, seed):
    c = case
    if c["kind"] in ("fork", "compact"):                 # (nothing is computed: pages and whole numbers)
        return None
    st = prepare(case, seed)
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    dev = st["q"].device
    if c["kind"] == "rope":
        pos = (c["start"] + torch.arange(c["L"], device=dev)).expand(c["B"], c["L"])
        return [_turned(st[n], pos, st["inv"], c["inter"], s) for n, s in (("q", 1), ("k", 1), ("dq", -1), ("dk", -1))]
    qs, kvs = ([], []) if c["kind"] == "train" else _lengths(c)
    if c["kind"] == "step":
        pos = torch.cat([torch.arange(kv, kv + n, device=dev) for n, kv in zip(qs, kvs)])
        k = st["k_cache"].double()
        at = torch.tensor(_places(c, st["table"].tolist(), k.shape[0], qs, kvs), device=dev).view(-1, 2)
        k[at[:, 0], at[:, 1]] = _turned(st["k_new"], pos, st["inv"], c["inter"], 1)
        return [_turned(st["q"], pos, st["inv"], c["inter"], 1), k] + [None] * 4
    W, ns = c["window"], c["sinks"]
    if c["kind"] == "paged":
        q, out, row = st["q"].double(), [], 0
        for b, (n, kv) in enumerate(zip(qs, kvs)):
            for t0 in range(0, n, 256):
                t1 = min(n, t0 + 256)
                pos = _exact_keys(kv + t0, kv + t1, W, ns, dev)
                pg = st["table"][b][pos // c["page"]].long()
                k, v = (st[x][pg, pos % c["page"]].double() for x in ("k_cache", "v_cache"))
                w, _, _, _, vv = _exact_rows(q[row + t0:row + t1], k, v, kv + t0, pos, c, st["slopes"])
                out.append(torch.einsum("hms,shd->mhd", w, vv))
            row += n
        return [torch.cat(out) if out else q.new_zeros(0, H, d)]
    B, L = c["B"], c["L"]
    o = torch.empty(B, L, H, d, device=dev, dtype=torch.float64)
    lse = torch.empty(B, L, H, device=dev, dtype=torch.float64)
    dq = torch.empty_like(o)
    dk = torch.zeros(B, L, Hkv, d, device=dev, dtype=torch.float64)
    dv = torch.zeros_like(dk)
    step = max(128, min(2048, W))
    for b in range(B):
        for t0 in range(0, L, step):
            t1 = min(L, t0 + step)
            pos = _exact_keys(t0, t1, W, ns, dev)
            q, k, v = st["q"][b, t0:t1].double(), st["k"][b, pos].double(), st["v"][b, pos].double()
            w, ls, turn, kk, vv = _exact_rows(q, k, v, t0, pos, c, st["slopes"])
            o[b, t0:t1] = torch.einsum("hms,shd->mhd", w, vv)
            lse[b, t0:t1] = ls.transpose(0, 1)
            g = st["dout"][b, t0:t1].double()
            dw = torch.einsum("mhd,shd->hms", g, vv)
            dz = w * (dw - (w * dw).sum(-1, keepdim=True)) * turn
            dq[b, t0:t1] = torch.einsum("hms,shd->mhd", dz, kk)
            fold = lambda x: x.view(len(pos), Hkv, H // Hkv, d).sum(2)  # noqa: E731
            dk[b].index_add_(0, pos, fold(torch.einsum("hms,mhd->shd", dz, q)))
            dv[b].index_add_(0, pos, fold(torch.einsum("hms,mhd->shd", w, g)))
    return [o, lse, dq, dk, dv]
