"""The pages of a paged cache on the GPU against a program on Python lists, and a generation that uses
all of it: reservation, turned writes, attention with transformed scores, forks, compaction."""
import random

import pytest
import torch

from retrieval_sparse_attention_gb300 import api

import score_reference as ref
from page_model import Pages
from test_gpu_rope import reference as turned

pytestmark = pytest.mark.gpu


class Device:
    """The same state on the GPU."""

    def __init__(self, m):
        self.m = m
        self.table = torch.tensor(m.table, dtype=torch.int32).cuda()
        self.kv = torch.tensor(m.kv, dtype=torch.int32).cuda()
        self.pool = api.page_pool(m.n)
        if any(m.refs):
            refs = torch.tensor(m.refs, dtype=torch.int32)
            bits = [0] * (-(-m.n // 32))
            for p in m.free():
                bits[p // 32] |= 1 << (p % 32)
            bits = torch.tensor([b - (1 << 32) if b >> 31 else b for b in bits], dtype=torch.int32)
            self.pool[:m.n], self.pool[m.n:m.n + bits.numel()] = refs.cuda(), bits.cuda()

    def check(self):
        m = self.m
        assert self.table.tolist() == m.table
        assert self.kv.tolist() == m.kv
        assert self.pool[:m.n].tolist() == m.refs
        words = self.pool[m.n:m.n + -(-m.n // 32)].tolist()
        assert [p for p in range(m.n) if words[p // 32] >> (p % 32) & 1] == m.free()
        assert all(not words[-1] >> i & 1 for i in range(m.n % 32 or 32, 32))
        assert api.gca_get_status() == m.status
        m.status = 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("B,width,n_pages,page,seed", [(1, 1, 1, 16, 0), (5, 8, 24, 16, 1), (40, 70, 1500, 16, 2), (7, 40, 100, 32, 3),
                                                       (300, 9, 1300, 16, 4), (3, 300, 33, 128, 5), (64, 20, 2000, 64, 6),
                                                       (70, 101, 4000, 16, 7), (4096, 1, 3000, 16, 8), (4096, 3, 9000, 16, 9)])
def test_any_sequence_of_calls(B, width, n_pages, page, seed):
    r = random.Random(seed)
    m = Pages(B, width, n_pages, page)
    s = Device(m)
    s.check()
    for _ in range(40):
        kind = r.randrange(6)
        if kind < 3:
            cu = [0]
            most = r.choice([1, 3, page + 3, width * page // 3])
            for _ in range(B):
                cu.append(cu[-1] + r.choice([0, 1, 1, 1, r.randint(0, most)]))
            window, sinks = r.choice([(0, 0), (1, 0), (page, 3), (2 * page + 5, page), (width * page // 2 + 1, page + 1), (2 ** 40, 1)])
            m.reserve(cu, window, sinks)
            api.paged_reserve(s.table, ints(cu), s.kv, s.pool, page=page, window=window, sinks=sinks)
        elif kind < 5:
            few = r.random() < 0.5                       # beams that change places, or sequences that end
            parent = [r.randrange(B) if r.random() < (0.1 if few else 0.6) else -1 if r.random() < 0.3 else b for b in range(B)]
            pairs = m.fork(parent)
            got = api.paged_fork(s.table, s.kv, ints(parent), s.pool, page=page)
            assert [tuple(x) for x in got.tolist()] == pairs
        else:
            n = r.choice([1, 2, n_pages])
            pairs = m.compact(n)
            got = api.paged_compact(s.table, s.pool, max_moves=n)
            assert [tuple(x) for x in got.tolist()] == pairs
        s.check()


def test_forks_of_sequences_that_were_set_back():
    # pages behind the length: one child keeps them, and no two write the same page afterwards
    m = Pages(5, 8, 40, 16)
    s = Device(m)
    m.reserve([0, 100, 100, 150, 150, 200])
    api.paged_reserve(s.table, ints([0, 100, 100, 150, 150, 200]), s.kv, s.pool, page=16)
    for lens in ([20, 0, 32, 0, 50], [5, 0, 1, 0, 16]):
        m.kv = list(lens)
        s.kv.copy_(ints(lens))
        for parent in ([0, 0, 2, 2, 0], [1, 0, 0, 2, 4]):
            pairs = m.fork(parent)
            got = api.paged_fork(s.table, s.kv, ints(parent), s.pool, page=16)
            assert [tuple(x) for x in got.tolist()] == pairs
            s.check()
        cu = [0, 30, 60, 90, 120, 150]
        m.reserve(cu)
        api.paged_reserve(s.table, ints(cu), s.kv, s.pool, page=16)
        s.check()
        for b, n in enumerate(m.kv):                     # what a sequence writes next it holds alone
            assert n < 0 or n % 16 == 0 or m.refs[m.table[b][n // 16]] == 1


def test_contradicting_arguments_are_reported():
    m = Pages(4, 4, 20, 16)
    s = Device(m)
    for cu in ([0, 3, 2, 10, 11], [0, 65, 66, 67, 68], [-1, 1, 2, 3, 4]):
        m.reserve(cu)
        api.paged_reserve(s.table, ints(cu), s.kv, s.pool, page=16)
        s.check()
    m.reserve([0, 1, 2, 3, 4])                           # those left out are taken up again
    api.paged_reserve(s.table, ints([0, 1, 2, 3, 4]), s.kv, s.pool, page=16)
    s.check()
    assert min(m.kv) >= 0
    for parent in ([0, 4, -2, 3], [2 ** 31 - 1, -2 ** 31, 0, 0]):
        pairs = m.fork(parent)
        got = api.paged_fork(s.table, s.kv, ints(parent), s.pool, page=16)
        assert [tuple(x) for x in got.tolist()] == pairs
        s.check()


def test_a_sequence_that_is_left_out_is_not_written():
    # too few pages: the length says so, and append and attention leave the sequence alone
    m = Pages(2, 4, 3, 16)
    s = Device(m)
    cu = ints([0, 30, 50])                               # two pages, and two of one
    api.paged_reserve(s.table, cu, s.kv, s.pool, page=16)
    assert s.kv.tolist() == [30, -1] and api.gca_get_status() == 7
    kc, vc = (torch.zeros(3, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = torch.ones(50, 1, 64, dtype=torch.bfloat16, device="cuda")
    api.paged_append(x, x, kc, vc, s.table, cu, s.kv)
    assert api.gca_get_status() == 6 and int((kc != 0).sum()) == 30 * 64
    out = torch.full_like(x, 5.0)
    api.paged_attn(x, kc, vc, s.table, cu, s.kv, out=out)
    assert api.gca_get_status() == 6 and (out[30:] == 5).all() and (out[:30] != 5).all()


@pytest.mark.parametrize("n_pages", [31, 32, 33, 1000, 40000, 1 << 20])
def test_a_pool_of_any_size(n_pages):
    pool = api.page_pool(n_pages)
    table = torch.full((1, 2048), -1, dtype=torch.int32, device="cuda")
    kv = ints([0])
    # the last pages alone are free
    words = -(-n_pages // 32)
    pool[:n_pages - 3] = 1
    pool[n_pages - 3:n_pages] = 0
    free = torch.zeros(words, 32, dtype=torch.int64)
    free.view(-1)[n_pages - 3:n_pages] = 1
    w = (free << torch.arange(32)).sum(1)
    pool[n_pages:n_pages + words] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).cuda()
    api.paged_reserve(table, ints([0, 33]), kv, pool, page=16)
    assert api.gca_get_status() == 0 and kv.tolist() == [33]
    assert table[0, :4].tolist() == [n_pages - 3, n_pages - 2, n_pages - 1, -1]
    assert int(pool[n_pages:n_pages + words].abs().max()) == 0
    if n_pages < 100000:
        pool[:n_pages - 3] = 0                           # those of others go: three are in use, at the end
        full = torch.ones(words, 32, dtype=torch.int64)
        full.view(-1)[n_pages - 3:] = 0
        w = (full << torch.arange(32)).sum(1)
        pool[n_pages:n_pages + words] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).cuda()
        pairs = api.paged_compact(table, pool, max_moves=5)
        assert pairs.tolist() == [[n_pages - 1, 0], [n_pages - 2, 1], [n_pages - 3, 2], [-1, -1], [-1, -1]]
        assert table[0, :4].tolist() == [2, 1, 0, -1]
        assert pool[:n_pages].tolist() == [1, 1, 1] + [0] * (n_pages - 3)


@pytest.mark.parametrize("shape,dtype", [((9, 16, 2, 64), torch.bfloat16), ((9, 128, 8, 128), torch.bfloat16), ((9, 16, 1, 8), torch.bfloat16),
                                         ((9, 4), torch.float32), ((9, 20, 3, 64), torch.float32)])
def test_copies(shape, dtype):
    k, v = (torch.randn(shape, device="cuda").to(dtype) for _ in range(2))
    a, b = k.clone(), v.clone()
    pairs = [(0, 3), (-1, -1), (0, 5), (8, 1), (-2, -2), (4, 4), (-1, 2), (2, -1)]
    api.paged_copy(k, v, ints(pairs))
    assert api.gca_get_status() == 0
    for src, dst in pairs:
        if src >= 0 and dst >= 0:
            a[dst], b[dst] = a[src].clone(), b[src].clone()
    assert torch.equal(a, k) and torch.equal(b, v)
    api.paged_copy(k, v, ints([(9, 0), (0, 9), (1, 2 ** 31 - 1)]))
    assert api.gca_get_status() == 6 and torch.equal(a, k) and torch.equal(b, v)
    api.paged_copy(k, v, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        api.paged_copy(k, v[:, :1], ints([(0, 1)]))
    with pytest.raises(ValueError):
        api.paged_copy(k, v, ints([0, 1]))


def test_binding_refusals():
    m = Pages(2, 4, 8, 16)
    s = Device(m)
    cu = ints([0, 1, 2])
    for bad in (dict(cu=cu[:2]), dict(kv=s.kv[:1]), dict(kv=s.kv.long()), dict(table=s.table.t()), dict(pool=s.pool[:-1]),
                dict(table=s.table.cpu())):
        a = dict(table=s.table, cu=cu, kv=s.kv, pool=s.pool, **{})
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            api.paged_reserve(a["table"], a["cu"], a["kv"], a["pool"], page=16)
    with pytest.raises(ValueError):
        api.paged_fork(s.table, s.kv, ints([0]), s.pool, page=16)
    with pytest.raises(ValueError):
        api.paged_compact(s.table, s.pool, max_moves=0)
    with pytest.raises(api.GcaError):
        api.paged_reserve(s.table, cu, s.kv, s.pool, page=24)
    s.check()


# --- a generation ------------------------------------------------------------------------
class Generation:
    """Tokens as each sequence has seen them, on the host, beside the device's cache."""

    def __init__(self, B, H, Hkv, d, page, n_pages, width, window, sinks, score, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.Hkv, self.d, self.page = B, H, Hkv, d, page
        self.window, self.sinks, self.score = window, sinks, score
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.kv = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.pool = api.page_pool(n_pages)
        self.kc, self.vc = (torch.full((n_pages, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.freqs = api.rope_freqs(d)
        self.k = [torch.zeros(0, Hkv, d) for _ in range(B)]
        self.v = [torch.zeros(0, Hkv, d) for _ in range(B)]

    def step(self, new):
        T = sum(new)
        q, k, v = (torch.randn(T, h, self.d, generator=self.g).to(torch.bfloat16) for h in (self.H, self.Hkv, self.Hkv))
        cu = ints([0] + new).cumsum(0).to(torch.int32)
        api.paged_reserve(self.table, cu, self.kv, self.pool, page=self.page, window=self.window, sinks=self.sinks)
        turned_q = api.paged_rope_append(q.cuda(), k.cuda(), v.cuda(), self.freqs, self.kc, self.vc, self.table, cu, self.kv)
        kw = {n: x.cuda() if torch.is_tensor(x) else x for n, x in self.score.items()}
        o, lse = api.paged_attn(turned_q, self.kc, self.vc, self.table, cu, self.kv, max_q=max(new), window=self.window,
                                sinks=self.sinks, with_lse=True, **kw)
        assert api.gca_get_status() == 0
        at = 0
        for b, n in enumerate(new):
            p0 = len(self.k[b])
            pos = torch.arange(p0, p0 + n)
            # keys as the cache holds them: turned in 64 bits, rounded once (the kernel's rounding of a value on a
            # border may fall on the other side: the cache's own rows are compared below, then used)
            kt, mag = turned(k[at:at + n], self.freqs, pos, False)
            rows = [(int(self.table[b, p // self.page]), p % self.page) for p in pos.tolist()]
            held = torch.stack([self.kc[i, j] for i, j in rows]).double().cpu() if n else kt
            assert ((held - kt).abs() <= 2.0 ** -8 * kt.abs() + 2.0 ** -20 * mag).all()
            self.k[b] = torch.cat([self.k[b].double(), held])
            self.v[b] = torch.cat([self.v[b].double(), v[at:at + n].double()])
            if n:
                cap, slopes = self.score.get("softcap", 0.0), self.score.get("slopes")
                ro, rl, bo, bl = ref.rows(turned_q[at:at + n].cpu(), self.k[b], self.v[b], pos, torch.arange(p0 + n), self.window,
                                          self.sinks, cap, slopes)
                ref.within("o of sequence %d" % b, o[at:at + n], ro, bo)
                ref.within("lse of sequence %d" % b, lse[at:at + n], rl, bl)
            at += n

    def fork(self, parent):
        pairs = api.paged_fork(self.table, self.kv, ints(parent), self.pool, page=self.page)
        api.paged_copy(self.kc, self.vc, pairs)
        assert api.gca_get_status() == 0
        none = torch.zeros(0, self.Hkv, self.d)
        self.k, self.v = ([x[p] if p >= 0 else none for p in parent] for x in (self.k, self.v))

    def compact(self):
        api.paged_copy(self.kc, self.vc, api.paged_compact(self.table, self.pool, max_moves=self.kc.shape[0]))
        used = int((self.pool[:self.kc.shape[0]] > 0).sum())
        assert int(self.table.max()) < used              # all at the front: what lies behind is cut off
        self.kc[used:] = float("nan")
        self.vc[used:] = float("nan")


@pytest.mark.parametrize("window,sinks,score", [(0, 0, dict(softcap=4.0)), (40, 3, dict(slopes=2.0 ** -torch.arange(1.0, 5.0))),
                                                (33, 20, dict())])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_generation(window, sinks, score, d, page):
    t = Generation(6, 4, 2, d, page, 120, 12, window, sinks, score, seed=d + window)
    t.step([50, 1, 0, 17, page, 0])                      # prompts, idle slots
    for _ in range(4):
        t.step([1, 1, 0, 1, 1, 0])
    t.fork([0, 0, 0, 3, 4, 3])                           # beams of two requests
    for _ in range(6):
        t.step([1, 1, 1, 1, 1, 1])
    t.fork([2, 1, 1, 5, -1, 3])                          # beams change places, a request ends
    t.step([1, 1, 1, 1, 30, 1])                          # another takes its slot
    t.compact()
    for _ in range(5):
        t.step([1, 1, 1, 1, 1, 1])
    t.fork([-1] * 6)
    n = t.kc.shape[0]
    assert int(t.pool[:n].abs().max()) == 0 and (t.table == -1).all()


def test_a_captured_generation():
    # reservation, write and attention in one graph, replayed: pages are taken and let go on the device
    B, H, Hkv, d, page, window, sinks = 5, 4, 2, 64, 16, 50, 4
    gen = torch.Generator().manual_seed(2)
    n_pages, width = 60, 40
    kv0 = [0, 15, 16, 47, 100]
    cu1 = ints([0] + kv0).cumsum(0).to(torch.int32)
    x = [torch.randn(sum(kv0), h, d, generator=gen).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv)]
    q, k, v = (torch.randn(60, B, h, d, generator=gen).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv))
    freqs, cu = api.rope_freqs(d), torch.arange(B + 1, dtype=torch.int32, device="cuda")

    class State:
        def __init__(self):
            self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
            self.kv = torch.zeros(B, dtype=torch.int32, device="cuda")
            self.pool = api.page_pool(n_pages)
            self.kc, self.vc = (torch.zeros(n_pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.q, self.k, self.v = (torch.empty(B, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
            self.out = torch.empty_like(self.q)
            self.run(cu1, *x)

        def run(self, cu, q, k, v):
            api.paged_reserve(self.table, cu, self.kv, self.pool, page=page, window=window, sinks=sinks)
            return api.paged_rope_append(q, k, v, freqs, self.kc, self.vc, self.table, cu, self.kv)

        def step(self):
            t = self.run(cu, self.q, self.k, self.v)
            api.paged_attn(t, self.kc, self.vc, self.table, cu, self.kv, max_q=1, window=window, sinks=sinks, softcap=5.0, out=self.out)

        def set(self, i):
            for a, b in ((self.q, q), (self.k, k), (self.v, v)):
                a.copy_(b[i])

    eager, graph = State(), State()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                           # (a step on each first: what is set up once is)
        for st in (eager, graph):
            st.set(0)
            st.step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step()
    for i in range(1, 60):
        eager.set(i)
        eager.step()
        graph.set(i)
        g.replay()
        for a, b in ((eager.out, graph.out), (eager.table, graph.table), (eager.kv, graph.kv)):
            assert torch.equal(a, b), i
    assert api.gca_get_status() == 0
    assert eager.kv.tolist() == [n + 60 for n in kv0]
    # pages behind the window came back: the sequences hold a window each
    assert int((eager.pool[:n_pages] > 0).sum()) <= B * (window // page + 3)


def test_copies_beyond_32_bits():
    # 2.6e9 elements of a cache: pages at its end
    n, shape = 20000, (128, 8, 128)
    k = torch.zeros(n, *shape, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    x, y = (torch.randn(shape, device="cuda").to(torch.bfloat16) for _ in range(2))
    k[n - 1], v[n - 2] = x, y
    api.paged_copy(k, v, ints([(n - 1, 3), (n - 2, n - 3)]))
    assert api.gca_get_status() == 0
    assert torch.equal(k[3], x) and torch.equal(v[n - 3], y) and not v[3].any() and not k[n - 3].any() and not k[4].any()
