"""The paged K/V cache: gca_paged_append and gca_paged_attn on the GPU against the
64-bit reference, on batches with idle slots, single tokens and chunks."""
import pytest
import torch

from retrieval_sparse_attention_gb300 import api
from retrieval_sparse_attention_gb300._lib import GcaError

import sink_reference as ref

pytestmark = pytest.mark.gpu

BAD_INDEX = 6


class Cache:
    """A cache with shuffled pages, NaN where nothing was written, and its sequences' tokens."""

    def __init__(self, qs, kvs, H, Hkv, d, page, seed=0, width=None, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.qs, self.kvs, self.H, self.Hkv, self.d, self.page = qs, kvs, H, Hkv, d, page
        need = [-(-n // page) for n in kvs]
        self.n_pages = sum(need) + spare
        ids = torch.randperm(self.n_pages, generator=g).tolist()
        width = max(max(need), 1) if width is None else width
        self.table = torch.full((len(qs), width), -1, dtype=torch.int32)
        shape = (self.n_pages, page, Hkv, d)
        self.kc = torch.full(shape, float("nan")).to(torch.bfloat16)
        self.vc = torch.full(shape, float("nan")).to(torch.bfloat16)
        self.k, self.v = [], []
        for b, n in enumerate(kvs):
            k, v = (torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
            self.k.append(k)
            self.v.append(v)
            for i in range(need[b]):
                pg = ids.pop()
                self.table[b, i] = pg
                part = slice(i * page, min(n, (i + 1) * page))
                self.kc[pg, :part.stop - part.start] = k[part]
                self.vc[pg, :part.stop - part.start] = v[part]
        self.cu = torch.tensor([0] + qs).cumsum(0).to(torch.int32)
        self.kv = torch.tensor(kvs, dtype=torch.int32)
        self.q = torch.randn(sum(qs), H, d, generator=g).to(torch.bfloat16)

    def cuda(self):
        return [x.cuda() for x in (self.q, self.kc, self.vc, self.table, self.cu, self.kv)]

    def check(self, o, lse, window, sinks, skip=()):
        for b, (n, kv) in enumerate(zip(self.qs, self.kvs)):
            if n == 0 or b in skip:
                continue
            rows = slice(int(self.cu[b]), int(self.cu[b + 1]))
            kpos = torch.arange(kv)
            ro, rl, bo, bl = ref.rows(self.q[rows], self.k[b], self.v[b], torch.arange(kv - n, kv), kpos, window,
                                      sinks) if kv else (torch.zeros(n, self.H, self.d).double(),
                                                         torch.full((n, self.H), float("-inf")).double(),
                                                         torch.zeros(n, self.H, self.d).double(), torch.zeros(n, self.H))
            ref.within("o of sequence %d" % b, o[rows], ro, bo)
            if lse is not None:
                ref.within("lse of sequence %d" % b, lse[rows], rl, bl)


# new tokens and lengths of a batch; H, Hkv, d, page; window, sinks
BATCHES = [([1], [1], 1, 1, 64, 16, 0, 0), ([1], [777], 12, 12, 64, 64, 512, 4), ([1, 1, 1], [5, 128, 129], 4, 2, 128, 32, 0, 0),
           ([1, 0, 3, 40, 0, 1], [300, 50, 3, 100, 0, 17], 6, 2, 64, 16, 64, 4),
           ([130, 1, 257], [130, 1000, 700], 4, 4, 64, 128, 0, 0), ([200], [900], 8, 1, 128, 64, 100, 16),
           ([33, 5], [33, 4000], 3, 1, 64, 64, 129, 33), ([1] * 20, list(range(1, 400, 20)), 8, 1, 64, 16, 0, 0),
           ([2, 1], [600, 601], 128, 1, 64, 32, 30, 1), ([70], [3000], 5, 1, 128, 64, 0, 0),
           ([1], [2500], 2, 2, 64, 16, 40, 1000), ([300, 0], [2000, 9], 2, 1, 64, 32, 1000, 2),
           ([1, 1], [1, 2], 24, 8, 128, 64, 1, 0), ([5] * 7, [5, 6, 7, 64, 65, 127, 250], 40, 1, 128, 16, 9, 3)]


@pytest.mark.parametrize("qs,kvs,H,Hkv,d,page,window,sinks", BATCHES)
def test_every_element(qs, kvs, H, Hkv, d, page, window, sinks):
    c = Cache(qs, kvs, H, Hkv, d, page, seed=sum(kvs))
    for max_q in (0, max(qs)):
        o, lse = api.paged_attn(*c.cuda(), max_q=max_q, window=window, sinks=sinks, with_lse=True)
        torch.cuda.synchronize()
        assert api.gca_get_status() == 0
        c.check(o, lse, window, sinks)


@pytest.mark.parametrize("qs,kvs,H,Hkv,d,page,window,sinks", [
    ([1, 1], [2000, 900], 16, 4, 128, 64, 600, 16), ([1, 1, 1], [5000, 4900, 130], 6, 6, 64, 16, 1500, 4),
    ([1, 2], [4000, 1000], 8, 2, 64, 32, 3000, 130), ([300, 1], [4000, 4000], 12, 12, 64, 64, 2500, 4)])
def test_windows_whose_units_are_cut(qs, kvs, H, Hkv, d, page, window, sinks):
    c = Cache(qs, kvs, H, Hkv, d, page, seed=sum(kvs))
    o, lse = api.paged_attn(*c.cuda(), max_q=max(qs), window=window, sinks=sinks, with_lse=True)
    assert api.gca_last_launch_count() == 2                # the join too
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    c.check(o, lse, window, sinks)


def test_long_cache_split_over_the_machine():
    # one token over a long cache, and a chunk beside it: the key axis is divided and joined
    c = Cache([1, 3, 1], [30000, 9000, 70], 4, 2, 128, 64, seed=1)
    o, lse = api.paged_attn(*c.cuda(), max_q=3, with_lse=True)
    c.check(o, lse, 0, 0)
    o2, lse2 = api.paged_attn(*c.cuda(), max_q=3, with_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H,Hkv,d,page,window,sinks", [(8, 2, 128, 64, 0, 0), (12, 12, 64, 16, 512, 4),
                                                       (6, 2, 64, 128, 700, 40), (4, 4, 128, 32, 100, 1)])
def test_serving_batch(H, Hkv, d, page, window, sinks):
    # many sequences of all kinds together: shares of many units, whole and cut
    g = torch.Generator().manual_seed(d + page)
    n = 40
    qs = [int(x) for x in torch.tensor([0, 1, 1, 1, 7, 130, 300, 513])[torch.randint(8, (n,), generator=g)]]
    kvs = [max(q, int(x)) for q, x in zip(qs, torch.randint(1, 3000, (n,), generator=g))]
    c = Cache(qs, kvs, H, Hkv, d, page, seed=7)
    o, lse = api.paged_attn(*c.cuda(), max_q=513, window=window, sinks=sinks, with_lse=True)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    c.check(o, lse, window, sinks)


def test_tokens_before_the_first_position_see_nothing():
    c = Cache([5, 4], [3, 0], 2, 1, 64, 16)
    o, lse = api.paged_attn(*c.cuda(), with_lse=True)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    c.check(o, lse, 0, 0)
    assert (o[:2] == 0).all() and torch.isneginf(lse[:2]).all() and (o[5:] == 0).all()


def test_rows_behind_the_last_sequence_stay():
    c = Cache([3, 2], [40, 9], 2, 2, 64, 16)
    q, kc, vc, table, cu, kv = c.cuda()
    pad = torch.full((4, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = torch.full((9, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    o, _ = api.paged_attn(torch.cat([q, pad]), kc, vc, table, cu, kv, out=out)
    assert o.data_ptr() == out.data_ptr()
    c.check(o, None, 0, 0)
    assert (o[5:] == 3.0).all()


def test_pages_that_left_the_window_are_not_looked_up():
    # as after their release: ids of nowhere, or pages full of NaN
    c = Cache([4, 1], [900, 640], 4, 2, 64, 16)
    gone = {}
    for b in range(2):
        first = c.kvs[b] - c.qs[b] - 100 + 1          # first key in the window of the first new token
        for i in range(1, first // 16):               # page 0 holds the sinks
            gone[(b, i)] = int(c.table[b, i])
            c.table[b, i] = [-1, 10 ** 9, c.n_pages][i % 3]
    assert len(gone) > 40
    o, lse = api.paged_attn(*c.cuda(), window=100, sinks=4, with_lse=True)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    c.check(o, lse, 100, 4)


@pytest.mark.parametrize("qs,kvs,H,Hkv,d,page,window,sinks", [b for b in BATCHES if b[6]] + [
    ([1, 9], [1300, 700], 4, 2, 128, 128, 200, 130), ([1, 1], [5000, 400], 12, 12, 64, 128, 300, 0),
    ([260, 1], [4000, 90], 2, 1, 128, 16, 65, 7), ([1, 0], [129, 40], 2, 2, 64, 64, 1, 0)])
def test_cache_rows_that_no_new_token_sees_may_hold_anything(qs, kvs, H, Hkv, d, page, window, sinks):
    # rows between the sinks and the first new token's window, in pages that hold visible rows too
    c = Cache(qs, kvs, H, Hkv, d, page, seed=sum(kvs))
    hidden = 0
    for b, (n, kv) in enumerate(zip(qs, kvs)):
        for s in range(min(sinks, kv), max(kv - n - window + 1, 0)) if n else range(kv):
            for x, bad in ((c.kc, float("nan")), (c.vc, [float("nan"), float("inf")][s % 2])):
                x[c.table[b, s // page], s % page] = bad
            hidden += 1
    assert hidden
    o, lse = api.paged_attn(*c.cuda(), max_q=max(qs), window=window, sinks=sinks, with_lse=True)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    c.check(o, lse, window, sinks)


def test_pages_may_be_shared():
    # three sequences with the same first pages, and a page that stands twice in one table row
    c = Cache([1, 5, 40], [200, 300, 170], 4, 2, 64, 16, seed=3)
    for b in (1, 2):
        c.table[b, :6] = c.table[0, :6]
        c.k[b][:96], c.v[b][:96] = c.k[0][:96], c.v[0][:96]
    c.table[1, 9] = c.table[1, 7]
    c.k[1][144:160], c.v[1][144:160] = c.k[1][112:128], c.v[1][112:128]
    for window, sinks in ((0, 0), (90, 20)):
        o, lse = api.paged_attn(*c.cuda(), window=window, sinks=sinks, with_lse=True)
        c.check(o, lse, window, sinks)
    assert api.gca_get_status() == 0


def test_rows_far_into_the_token_tensors():
    # the call's tokens are rows behind 2^26 others (32 lanes a row: past 32 bits of threads)
    c = Cache([3, 2], [40, 9], 1, 1, 64, 16, seed=5)
    q, kc, vc, table, cu, kv = c.cuda()
    first = 2 ** 26 + 1
    big = torch.empty(first + 6, 1, 64, dtype=torch.bfloat16, device="cuda")
    cu = cu + first
    big[first:first + 5] = q
    o, lse = api.paged_attn(big, kc, vc, table, cu, kv, max_q=3, with_lse=True)
    c.check(o[first:first + 5], lse[first:first + 5], 0, 0)
    kc.zero_()
    vc.zero_()
    api.paged_append(big, big, kc, vc, table, cu, kv, max_q=3)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    for row, (b, s) in enumerate([(0, 37), (0, 38), (0, 39), (1, 7), (1, 8)]):
        for x in (kc, vc):
            assert torch.equal(x[table[b, s // 16].item(), s % 16], big[first + row])
    assert int((kc.abs().sum(-1) > 0).sum()) == 5


@pytest.mark.parametrize("d,window", [(64, 900), (128, 500)])
def test_many_units_of_long_windows(d, window):
    # so many that the two workers of a CTA share one stretch of units: the same bits as from
    # calls on a few of the heads, dense and through the cache
    B, L, H, page = 2, 2600, 64, 64
    g = torch.Generator().manual_seed(d)
    q, k, v = (torch.randn(B, L, H, d, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    o, lse = api.swa_sink_fwd(q, k, v, window=window, sinks=4)
    assert api.gca_last_launch_count() == 1
    for h in (0, 31, 62):
        heads = slice(h, h + 2)
        a, b = api.swa_sink_fwd(*(x[:, :, heads].contiguous() for x in (q, k, v)), window=window, sinks=4)
        assert torch.equal(o[:, :, heads], a) and torch.equal(lse[:, :, heads], b)
    n = -(-L // page)
    table = torch.randperm(B * n, generator=g).view(B, n).to(torch.int32).cuda()
    kc, vc = (torch.full((B * n, page, H, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu = torch.tensor([0, L, 2 * L], dtype=torch.int32, device="cuda")
    kv = torch.tensor([L, L], dtype=torch.int32, device="cuda")
    api.paged_append(k.view(B * L, H, d), v.view(B * L, H, d), kc, vc, table, cu, kv)
    a, b = api.paged_attn(q.view(B * L, H, d), kc, vc, table, cu, kv, max_q=L, window=window, sinks=4, with_lse=True)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    assert torch.equal(a.view_as(o), o) and torch.equal(b.view_as(lse), lse)


def test_two_streams_at_once():
    # calls that overlap, each with its own workspace, and what they give one after the other
    a = Cache([1] * 8, [4000 + 300 * i for i in range(8)], 8, 2, 128, 64, seed=8)
    b = Cache([300, 20], [2500, 900], 12, 12, 64, 16, seed=9)
    ta, tb = a.cuda(), b.cuda()
    want = api.paged_attn(*ta, max_q=1, with_lse=True) + api.paged_attn(*tb, window=512, sinks=4, with_lse=True)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(sa):
            ga = api.paged_attn(*ta, max_q=1, with_lse=True)
        with torch.cuda.stream(sb):
            gb = api.paged_attn(*tb, window=512, sinks=4, with_lse=True)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ga + gb, want))
    assert api.gca_get_status() == 0


def test_a_bad_page_reads_as_zeros_and_is_reported():
    c = Cache([1, 2], [100, 200], 2, 1, 64, 32)
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        for b in (0,):
            c.table[b, 1] = bad
        k, v = c.k[0].clone(), c.v[0].clone()
        c.k[0][32:64] = 0
        c.v[0][32:64] = 0
        o, lse = api.paged_attn(*c.cuda(), with_lse=True)
        torch.cuda.synchronize()
        assert api.gca_get_status() == BAD_INDEX
        assert api.gca_get_status() == 0
        c.check(o, lse, 0, 0)
        c.k[0], c.v[0] = k, v


@pytest.mark.parametrize("what", ["cu_down", "cu_over", "cu_negative", "too_many", "kv_negative", "kv_over"])
def test_contradicting_lengths_leave_a_sequence_out(what):
    c = Cache([2, 3, 4], [40, 50, 60], 2, 1, 64, 16)
    q, kc, vc, table, cu, kv = c.cuda()
    max_q, skip = 4, (1,)
    if what == "cu_down":
        cu[2] = 1
        skip = (1, 2)                                 # sequence 2 now claims rows 1 .. 8: too many
    elif what == "cu_over":
        cu[3] = 10
        skip = (2,)
    elif what == "cu_negative":
        cu[0] = -1
        skip = (0,)
    elif what == "too_many":
        max_q, skip = 3, (2,)
    elif what == "kv_negative":
        kv[1] = -5
    else:
        kv[1] = table.shape[1] * 16 + 1
    out = torch.full((9, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    o, _ = api.paged_attn(q, kc, vc, table, cu, kv, max_q=max_q, out=out)
    torch.cuda.synchronize()
    assert api.gca_get_status() == BAD_INDEX
    c.check(o, None, 0, 0, skip=skip)
    for b in skip:
        assert (o[int(c.cu[b]):int(c.cu[b + 1])] == 3.0).all()
    kc2, vc2 = kc.clone(), vc.clone()
    kn = torch.randn(9, 1, 64, device="cuda").to(torch.bfloat16)
    api.paged_append(kn, kn, kc2, vc2, table, cu, kv, max_q=max_q)
    torch.cuda.synchronize()
    assert api.gca_get_status() == BAD_INDEX
    for b in range(3):
        for i in range(c.qs[b]):
            pos = c.kvs[b] - c.qs[b] + i
            got = kc2[int(c.table[b, pos // 16]), pos % 16]
            want = kc[int(c.table[b, pos // 16]), pos % 16] if b in skip else kn[int(c.cu[b]) + i]
            assert torch.equal(got, want)


@pytest.mark.parametrize("qs,kvs,Hkv,d,page", [([1, 0, 5, 33], [1, 7, 5, 100], 2, 64, 16), ([300], [700], 1, 128, 128),
                                               ([1] * 9, list(range(3, 30, 3)), 12, 64, 32), ([3, 2], [2, 2], 3, 64, 16)])
@pytest.mark.parametrize("max_q", [0, 1])
def test_append_writes_its_rows_and_no_others(qs, kvs, Hkv, d, page, max_q):
    c = Cache(qs, kvs, Hkv, Hkv, d, page, seed=3)
    _, kc, vc, table, cu, kv = c.cuda()
    T = sum(qs)
    x = torch.randn(T + 2, 2, Hkv, d).to(torch.bfloat16)          # k and v packed, two rows of padding
    want_k, want_v = c.kc.clone(), c.vc.clone()
    for b, n in enumerate(qs):
        for i in range(n):
            pos = kvs[b] - n + i
            if pos < 0:
                continue
            want_k[int(c.table[b, pos // page]), pos % page] = x[int(c.cu[b]) + i, 0]
            want_v[int(c.table[b, pos // page]), pos % page] = x[int(c.cu[b]) + i, 1]
    xc = x.cuda()
    api.paged_append(xc[:, 0], xc[:, 1], kc, vc, table, cu, kv, max_q=max(qs) if max_q else 0)
    torch.cuda.synchronize()
    assert api.gca_get_status() == 0
    same = lambda a, b: torch.equal(a.cpu().view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(kc, want_k) and same(vc, want_v)


def test_append_to_many_sequences():
    # far more than a warp looks at together, idle ones and chunks among single tokens
    g = torch.Generator().manual_seed(6)
    qs = [int(x) for x in torch.tensor([0, 1, 1, 1, 2, 0, 60])[torch.randint(7, (700,), generator=g)]]
    kvs = [q + int(x) for q, x in zip(qs, torch.randint(0, 50, (700,), generator=g))]
    test_append_writes_its_rows_and_no_others(qs, kvs, 2, 64, 16, 60)


def test_append_reports_a_bad_page_and_writes_the_rest():
    c = Cache([40], [40], 1, 1, 64, 16)
    c.table[0, 1] = c.n_pages
    _, kc, vc, table, cu, kv = c.cuda()
    x = torch.randn(40, 1, 64).to(torch.bfloat16)
    before = kc.clone()
    api.paged_append(x.cuda(), x.cuda(), kc, vc, table, cu, kv)
    torch.cuda.synchronize()
    assert api.gca_get_status() == BAD_INDEX
    kept = [int(c.table[0, 0]), int(c.table[0, 2])]
    assert torch.equal(kc[kept[0]].cpu(), x[:16]) and torch.equal(kc[kept[1], :8].cpu(), x[32:])
    rest = [i for i in range(c.n_pages) if i not in kept]
    assert torch.equal(kc[rest].view(torch.int16), before[rest].view(torch.int16))


def test_prompt_in_chunks_then_tokens():
    """As a server uses them: a prompt in two chunks beside another sequence's tokens, then
    single tokens, through the window; each output row is the one that the dense operator
    gives on the whole sequence."""
    H, Hkv, d, page, W, ns, n = 6, 2, 64, 16, 100, 4, 340
    g = torch.Generator().manual_seed(12)
    seq = [[torch.randn(n, h, d, generator=g).to(torch.bfloat16) for h in (H, Hkv, Hkv)] for _ in range(2)]
    q, k, v = (torch.stack([s[i] for s in seq]).cuda() for i in range(3))
    ro, rl, bo, bl = ref.forward(*(x.cpu() for x in (q, k, v)), W, ns)
    kc = torch.full((50, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    table = torch.randperm(50, generator=g)[:44].view(2, 22).to(torch.int32).cuda()
    done = [0, 0]
    steps = [(150, 1), (0, 1), (150, 30)] + [(1, 1)] * 20 + [(20, 3)]
    for step in steps:
        parts = [[x[b, done[b]:done[b] + m] for b, m in enumerate(step)] for x in (q, k, v)]
        qn, kn, vn = (torch.cat(p) for p in parts)
        cu = torch.tensor([0, step[0], sum(step)], dtype=torch.int32, device="cuda")
        kv = torch.tensor([done[b] + step[b] for b in range(2)], dtype=torch.int32, device="cuda")
        api.paged_append(kn, vn, kc, vc, table, cu, kv, max_q=max(step))
        o, lse = api.paged_attn(qn, kc, vc, table, cu, kv, max_q=max(step), window=W, sinks=ns, with_lse=True)
        row = 0
        for b, m in enumerate(step):
            at = slice(done[b], done[b] + m)
            ref.within("o", o[row:row + m], ro[b, at], bo[b, at])
            ref.within("lse", lse[row:row + m], rl[b, at], bl[b, at])
            row += m
            done[b] += m
        # pages that the window has left are given back
        for b in range(2):
            for i in range(1, max(0, done[b] - W + 1) // page):
                table[b, i] = -1
    assert api.gca_get_status() == 0 and done == [340, 55]


def test_captured_step_follows_the_lengths():
    """One captured append + attention, replayed as the sequences grow; two graphs with
    workspaces of their own, replayed on two streams."""
    H, Hkv, d, page, B = 4, 2, 64, 16, 3
    g = torch.Generator().manual_seed(2)
    total = 60
    q, k, v = (torch.randn(B, total, h, d, generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv))
    ro, rl, bo, bl = ref.forward(*(x.cpu() for x in (q, k, v)), total, 0)
    sets = []
    for _ in range(2):
        kc = torch.full((12, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        vc = kc.clone()
        table = torch.randperm(12, generator=g).view(3, 4).to(torch.int32).cuda()
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        kv = torch.ones(B, dtype=torch.int32, device="cuda")
        qn, kn, vn = q[:, 0].clone(), k[:, 0].clone(), v[:, 0].clone()
        api.paged_attn(qn, kc, vc, table, cu, kv, max_q=1)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.paged_append(kn, vn, kc, vc, table, cu, kv, max_q=1)
            o, _ = api.paged_attn(qn, kc, vc, table, cu, kv, max_q=1)
        sets.append((graph, qn, kn, vn, kv, o, torch.cuda.Stream(), kc, vc, table, cu))
    torch.cuda.synchronize()
    for t in range(total):
        for graph, qn, kn, vn, kv, o, stream, *_ in sets:
            with torch.cuda.stream(stream):
                qn.copy_(q[:, t])
                kn.copy_(k[:, t])
                vn.copy_(v[:, t])
                kv.fill_(t + 1)
                graph.replay()
        torch.cuda.synchronize()
        for s in sets:
            ref.within("o at %d" % t, s[5], ro[:, t], bo[:, t])


def test_offsets_past_32_bits():
    # the cache's last pages lie beyond 2^32 bytes and 2^31 elements
    page, Hkv, d, n_pages = 128, 8, 128, 17000
    kc = torch.zeros(n_pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() > 2 ** 31
    g = torch.Generator().manual_seed(5)
    n = 300
    k, v = (torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kv = torch.tensor([n], dtype=torch.int32, device="cuda")
    api.paged_append(k.cuda(), v.cuda(), kc, vc, table, cu, kv)
    o, lse = api.paged_attn(q.cuda(), kc, vc, table, cu, kv, with_lse=True)
    ro, rl, bo, bl = ref.rows(q, k, v, torch.arange(n), torch.arange(n), 0, 0)
    ref.within("o", o, ro, bo)
    ref.within("lse", lse, rl, bl)
    assert torch.equal(kc[n_pages - 1].cpu(), k[:128])


def test_nothing_to_do():
    c = Cache([0, 0], [5, 0], 2, 1, 64, 16)
    q, kc, vc, table, cu, kv = c.cuda()
    o, lse = api.paged_attn(q, kc, vc, table, cu, kv, with_lse=True)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    x = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    api.paged_append(x, x, kc, vc, table, cu, kv)
    # rows but no sequence that has any
    pad = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(pad, 2.0)
    api.paged_attn(pad, kc, vc, table, cu, kv, out=out)
    torch.cuda.synchronize()
    assert (out == 2.0).all() and api.gca_get_status() == 0


def test_refusals():
    c = Cache([1], [20], 2, 1, 64, 16)
    q, kc, vc, table, cu, kv = c.cuda()
    for bad in (dict(q=q.float()), dict(table=table.long()), dict(cu=cu.long()), dict(kv=kv.float()),
                dict(vc=vc.float())):
        a = dict(q=q, kc=kc, vc=vc, table=table, cu=cu, kv=kv)
        a.update(bad)
        with pytest.raises(TypeError):
            api.paged_attn(*a.values())
    for bad in (dict(q=q[:, :, :32]), dict(cu=cu[:1]), dict(kv=kv.repeat(2)), dict(vc=vc[:-1]), dict(table=table[0]),
                dict(q=q.cpu()), dict(kv=kv.cpu()), dict(kc=kc[:, ::2])):
        a = dict(q=q, kc=kc, vc=vc, table=table, cu=cu, kv=kv)
        a.update(bad)
        with pytest.raises(ValueError):
            api.paged_attn(*a.values())
    with pytest.raises(GcaError) as e:
        api.paged_attn(q, kc[:, :8].contiguous(), vc[:, :8].contiguous(), table, cu, kv)     # pages of 8 tokens
    assert e.value.code == 2
    with pytest.raises(GcaError) as e:
        api.paged_attn(q, kc, vc, table, cu, kv, window=-1)
    assert e.value.code == 1
    with pytest.raises(ValueError):
        api.paged_append(q, q, kc, vc, table, cu, kv)                                        # 2 heads, cache has 1
    with pytest.raises(ValueError):
        api.paged_attn(q, kc, vc, table, cu, kv, out=torch.empty(2, 2, 64, dtype=torch.bfloat16, device="cuda"))
