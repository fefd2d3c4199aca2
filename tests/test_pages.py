"""Upkeep of paged caches (append, reserve, fork, free, compact) against plain
lists, bit for bit, their refusals, and a run of all of them with attention."""
import math
import random

import pytest
import torch

from paged_reference import Pages, attention, check

FAKE = 0x10000


@pytest.fixture(scope="module")
def attn():
    from exact_softmax_attention_04_b200 import build_lib
    build_lib.build()
    import exact_softmax_attention_04_b200 as pkg
    return pkg


@pytest.fixture
def gpu(attn):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return attn


# ---------------------------------------------------------------- refusals

def strides(*s):
    import ctypes
    return (ctypes.c_int64 * len(s))(*s)


A = dict(k=FAKE, v=FAKE, ks=None, vs=None, kp=FAKE, vp=FAKE, ps=None, table=FAKE, pos=FAKE, count=0, B=2, Hkv=2, T=3,
         P=64, page=16, width=8, d=128, lens=FAKE, refs=FAKE, rows=FAKE, want=FAKE, granted=FAKE, ws=FAKE,
         ws_bytes=1 << 40, n=4, R=8, fresh=FAKE, tout=FAKE, rout=FAKE, live=FAKE)

POOLS = [(dict(kp=0), 1), (dict(kp=FAKE + 8), 1), (dict(vp=FAKE + 8), 1), (dict(Hkv=0), 1), (dict(P=0), 1),
         (dict(page=0), 1), (dict(d=0), 1), (dict(ps=strides(4096, 2048, 64)), 1), (dict(d=100), 2), (dict(d=1032), 2),
         (dict(P=1 << 21), 2), (dict(page=1 << 28), 2)]
STATE = [(dict(table=0), 1), (dict(refs=0), 1), (dict(table=FAKE + 2), 1), (dict(ws=0), 1), (dict(ws_bytes=8), 1),
         (dict(R=0), 1), (dict(width=0), 1)]


@pytest.mark.parametrize("kw,code", POOLS + [(dict(k=0), 1), (dict(v=0), 1), (dict(k=FAKE + 2), 1), (dict(B=0), 1),
                                             (dict(T=0), 1), (dict(pos=0), 1), (dict(count=FAKE + 1), 1),
                                             (dict(ks=strides(8, 8, 4)), 1), (dict(ks=strides(8, -8, 8)), 1),
                                             (dict(B=70000), 2), (dict(T=1 << 30), 2),
                                             (dict(Hkv=1 << 17, d=1024, page=1, T=1), 2)])
def test_append_refuses_before_any_cuda_call(attn, kw, code):
    a = A | kw
    assert attn.lib().attn_pages_append(a["k"], a["v"], a["ks"], a["vs"], a["kp"], a["vp"], a["ps"], a["table"],
                                        a["pos"], a["count"], a["B"], a["Hkv"], a["T"], a["P"], a["page"],
                                        a["width"], a["d"], None) == code


@pytest.mark.parametrize("kw,code", STATE + [(dict(rows=0), 1), (dict(want=0), 1), (dict(granted=0), 1),
                                             (dict(n=-1), 1), (dict(P=0), 1), (dict(page=0), 1), (dict(P=1 << 21), 2)])
def test_reserve_refuses_before_any_cuda_call(attn, kw, code):
    a = A | kw
    assert attn.lib().attn_pages_reserve(a["table"], a["refs"], a["rows"], a["want"], a["granted"], a["ws"],
                                         a["ws_bytes"], a["n"], a["R"], a["P"], a["page"], a["width"], None) == code


@pytest.mark.parametrize("kw,code", POOLS + STATE + [(dict(rows=0), 1), (dict(want=0), 1), (dict(fresh=0), 1),
                                                     (dict(granted=0), 1), (dict(lens=0), 1), (dict(n=-1), 1)])
def test_fork_refuses_before_any_cuda_call(attn, kw, code):
    a = A | kw
    assert attn.lib().attn_pages_fork(a["kp"], a["vp"], a["ps"], a["table"], a["lens"], a["refs"], a["rows"],
                                      a["want"], a["fresh"], a["granted"], a["ws"], a["ws_bytes"], a["n"], a["R"],
                                      a["Hkv"], a["P"], a["page"], a["width"], a["d"], None) == code


@pytest.mark.parametrize("kw", [dict(table=0), dict(lens=0), dict(refs=0), dict(rows=0), dict(n=-1), dict(R=0),
                                dict(P=0), dict(width=0), dict(rows=FAKE + 2)])
def test_free_refuses_before_any_cuda_call(attn, kw):
    a = A | kw
    assert attn.lib().attn_pages_free(a["table"], a["lens"], a["refs"], a["rows"], a["n"], a["R"], a["P"],
                                      a["width"], None) == 1


@pytest.mark.parametrize("kw,code", POOLS + STATE + [(dict(tout=0), 1), (dict(rout=0), 1), (dict(live=0), 1)])
def test_compact_refuses_before_any_cuda_call(attn, kw, code):
    a = A | kw
    assert attn.lib().attn_pages_compact(a["kp"], a["vp"], a["ps"], a["table"], a["refs"], a["tout"], a["rout"],
                                         a["live"], a["ws"], a["ws_bytes"], a["R"], a["Hkv"], a["P"], a["page"],
                                         a["width"], a["d"], None) == code


def test_no_requests_is_no_work(attn):
    lib = attn.lib()
    assert lib.attn_pages_reserve(FAKE, FAKE, 0, 0, 0, 0, 0, 0, 8, 64, 16, 8, None) == 0
    assert lib.attn_pages_free(FAKE, FAKE, FAKE, 0, 0, 8, 64, 8, None) == 0
    assert lib.attn_pages_fork(FAKE, FAKE, None, FAKE, FAKE, FAKE, 0, 0, 0, 0, 0, 0, 0, 8, 2, 64, 16, 8, 128, None) == 0


def test_workspace_size(attn):
    assert attn.pages_workspace_bytes(0, 1, 1) > 0
    for bad in [(-1, 8, 64), (1, 0, 64), (1, 8, 0), (1, 8, 1 << 21)]:
        with pytest.raises(ValueError):
            attn.pages_workspace_bytes(*bad)


def test_the_plain_lists_keep_their_counts():
    """The lists' own book-keeping: counts are the rows that hold a page."""
    rng = random.Random(3)
    book = Pages([[-1] * 6 for _ in range(10)], [0] * 10, [0] * 40, 4)
    for step in range(200):
        what = rng.choice(["reserve", "fork", "free", "compact"])
        rows = [rng.randrange(-1, 11) for _ in range(rng.randrange(1, 4))]
        if what == "reserve":
            want = [rng.randrange(0, 26) for _ in rows]
            for r, w, ok in zip(rows, want, book.reserve(rows, want)):
                if ok:
                    book.lens[r] = max(book.lens[r], w)
        elif what == "fork":
            book.fork(rows, [rng.randrange(0, 10) for _ in rows])
        elif what == "free":
            book.free(rows)
        else:
            book.compact()
        held = [0] * 40
        for row in book.table:
            for e in row:
                if e >= 0:
                    held[e] += 1
        assert held == book.refs


# ------------------------------------------------------------------ helpers

def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pools(P, Hkv, page, d, layout, seed):
    """One or two pools: contiguous, token-major, padded and interleaved, latent."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    if layout == "latent":
        return rnd(P, page, d), None
    if layout == "nhd":
        return rnd(P, page, Hkv, d).transpose(1, 2), rnd(P, page, Hkv, d).transpose(1, 2)
    if layout == "padded":
        both = rnd(P, 2, Hkv, page, d + 8)
        return both[:, 0, ..., :d], both[:, 1, ..., :d]
    return rnd(P, Hkv, page, d), rnd(P, Hkv, page, d)


def as4(x):
    return x.unsqueeze(1) if x.dim() == 3 else x


class Both:
    """The same state on the device and in lists."""

    def __init__(self, R, width, P, Hkv, page, d, layout, seed):
        self.k, self.v = pools(P, Hkv, page, d, layout, seed)
        self.table, self.lens = torch.full((R, width), -1, dtype=torch.int32, device="cuda"), int32([0] * R)
        self.refs = int32([0] * P)
        self.book = Pages(self.table, self.lens, self.refs, page)
        self.want = [x.clone() for x in self.pools()]
        self.page = page

    def pools(self):
        return [x for x in (self.k, self.v) if x is not None]

    def same(self):
        assert self.table.tolist() == self.book.table
        assert self.lens.tolist() == self.book.lens
        assert self.refs.tolist() == self.book.refs
        for x, y in zip(self.pools(), self.want):
            assert torch.equal(x.view(torch.int16) if x.is_contiguous() else x, y.view(torch.int16) if x.is_contiguous() else y)

    def set_lens(self, lens):
        self.lens.copy_(int32(lens))
        self.book.lens = list(lens)

    def reserve(self, attn, rows, want):
        got = attn.pages_reserve(self.table, self.refs, int32(rows), int32(want), self.page)
        assert got.tolist() == self.book.reserve(rows, want)
        self.same()
        return got.tolist()

    def fork(self, attn, parents, children):
        fresh, granted = attn.pages_fork(self.k, self.v, self.table, self.lens, self.refs, int32(parents),
                                         int32(children))
        f, ok, copies = self.book.fork(parents, children)
        for a, b, n in copies:
            for x in self.want:
                as4(x)[b, :, :n] = as4(x)[a, :, :n]
        assert fresh.tolist() == f and granted.tolist() == ok
        self.same()

    def free(self, attn, rows):
        attn.pages_free(self.table, self.lens, self.refs, int32(rows))
        self.book.free(rows)
        self.same()

    def compact(self, attn, in_place=True):
        out = None if in_place else (torch.full_like(self.table, 99), torch.full_like(self.refs, 99))
        before = (self.table.clone(), self.refs.clone())
        live = attn.pages_compact(self.k, self.v, self.table, self.refs, out=out)
        n, moves = self.book.compact()
        for a, b in moves:
            for x in self.want:
                x[b] = x[a]
        if out is not None:
            assert torch.equal(self.table, before[0]) and torch.equal(self.refs, before[1])
            self.table, self.refs = out
        assert live.tolist() == [n]
        self.same()


LAYOUTS = [("hnd", 2, 64), ("nhd", 3, 128), ("padded", 2, 64), ("latent", 1, 576), ("hnd", 1, 8)]


# -------------------------------------------------------------------- append

@pytest.mark.gpu
@pytest.mark.parametrize("layout,Hkv,d", LAYOUTS)
@pytest.mark.parametrize("page,T", [(1, 3), (8, 1), (12, 5), (16, 40), (64, 200)])
@pytest.mark.parametrize("source", ["hnd", "token-major", "shared"])
def test_append(gpu, layout, Hkv, d, page, T, source):
    B, width = 4, 1000 // page
    g = torch.Generator(device="cuda")
    g.manual_seed(page + T)
    k, v = pools(4 * width + 2, Hkv, page, d, layout, 1)
    table = torch.randperm(4 * width + 2, generator=g, device="cuda")[: 4 * width].int().view(4, width)
    table[1, 1], table[1, 2] = -1, 4 * width + 2
    pos, count = int32([0, page, 1000 - 2, -2]), int32([T, T + 9, T, max(T - 1, 0)])
    shape = {"hnd": (B, Hkv, T, d), "token-major": (B, T, Hkv, d), "shared": (1, Hkv, T, d)}[source]
    new = [torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2)]
    if source == "token-major":
        new = [x.transpose(1, 2) for x in new]
    if source == "shared":
        new = [x.expand(B, -1, -1, -1) for x in new]
    have = [x for x in (k, v) if x is not None]
    want = [x.clone() for x in have]
    for b in range(B):
        for u in range(min(max(int(count[b]), 0), T)):
            p = int(pos[b]) + u
            if 0 <= p < width * page and 0 <= int(table[b, p // page]) < 4 * width + 2:
                for x, y in zip(want, new):
                    as4(x)[int(table[b, p // page]), :, p % page] = y[b, :, u]
    gpu.pages_append(new[0], None if v is None else new[1], k, v, table, pos, count)
    torch.cuda.synchronize()
    for x, y in zip(have, want):
        assert torch.equal(x, y)
    if T == 5:  # every token
        gpu.pages_append(new[0][:1], None if v is None else new[1][:1], k, v, table[:1], pos[:1])
        for x, y in zip(want, new):
            for u in range(T):
                as4(x)[int(table[0, u // page]), :, u % page] = y[0, :, u]
        for x, y in zip(have, want):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_append_offsets_past_32_bits(gpu):
    P, Hkv, page, d = 34000, 8, 128, 128
    k = torch.zeros((P, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    new = torch.randn((2, Hkv, 3, d), device="cuda").bfloat16()
    table = int32([[P - 1], [33333]])
    gpu.pages_append(new, new, k, k, table, int32([0, 100]))
    assert torch.equal(k[P - 1, :, :3], new[0]) and torch.equal(k[33333, :, 100:103], new[1])
    assert int((k[::1000].float().abs().amax((1, 2, 3)) > 0).sum()) == 0


# ------------------------------------------------------- reserve, fork, free

@pytest.mark.gpu
@pytest.mark.parametrize("layout,Hkv,d", LAYOUTS)
@pytest.mark.parametrize("page", [1, 16, 20])
def test_fork_shares_and_copies(gpu, layout, Hkv, d, page):
    s = Both(12, 7, 60, Hkv, page, d, layout, 2)
    s.reserve(gpu, [0, 3, 5], [7 * page, 2 * page + 1, page])
    s.set_lens([7 * page - page // 2, 0, 0, 2 * page + 1, 0, page] + [0] * 6)
    s.fork(gpu, [0, 0, 3, 5, 1], [1, 7, 2, 11, 4])
    s.fork(gpu, [1, 2], [6, 8])
    s.free(gpu, [0, 1, 11])
    s.compact(gpu)
    s.reserve(gpu, [6, 0], [7 * page, 3])


@pytest.mark.gpu
def test_requests_that_cannot_be_met(gpu):
    s = Both(8, 6, 20, 2, 8, 64, "hnd", 3)
    assert s.reserve(gpu, [0, 1, -1, 8, 1, 2, 3], [48, 20, 8, 8, 8, 49, 0]) == [1, 1, 0, 0, 0, 0, 1]
    s.set_lens([45, 20, 0, 0, 0, 0, 0, 0])
    # out of range, twice the same child, a child with content, itself, a
    # parent that is another request's child
    s.fork(gpu, [0, 0, -1, 9, 1, 1, 4, 0], [2, 2, 3, 3, 0, 1, 5, 4])
    # 20 - 9 - 2 pages left: the third is refused, and what follows needs none
    assert s.reserve(gpu, [3, 5, 6, 7], [40, 32, 8, 0]) == [1, 1, 0, 1]
    s.fork(gpu, [1, 3], [6, 7])
    s.free(gpu, [2, 2, 100, -4, 0])
    s.reserve(gpu, [0], [48])
    s.free(gpu, list(range(8)))
    assert s.refs.tolist() == [0] * 20


@pytest.mark.gpu
def test_state_that_is_out_of_order(gpu):
    """Entries that are no page, counts below 0 and lengths beyond the table."""
    s = Both(6, 4, 30, 1, 8, 64, "hnd", 4)
    for r, row in enumerate([[3, 99, 5, 6], [7, -1, -1, -1], [-1, 8, -1, -1]]):
        s.table[r] = int32(row)
        s.book.table[r] = row
    for p, n in [(3, 1), (5, 1), (6, 1), (7, 2), (8, 1), (0, -2), (1, -1)]:
        s.refs[p] = n
        s.book.refs[p] = n
    s.set_lens([30, 33, 0, 0, 0, 0])
    s.fork(gpu, [0, 1, 0], [3, 4, 2])
    s.free(gpu, [3])
    s.compact(gpu)
    s.reserve(gpu, [2, 4], [32, 32])


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(4))
def test_random_runs(gpu, seed):
    rng = random.Random(seed)
    page, P = rng.choice([4, 16]), rng.choice([50, 5000])
    R, width = 40, 12
    layout, Hkv, d = rng.choice(LAYOUTS)
    s = Both(R, width, P, Hkv, page, d, layout, seed)
    for step in range(25):
        what = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        n = rng.randrange(1, 30)
        if what == "reserve":
            rows, want = [rng.randrange(R) for _ in range(n)], [rng.randrange(width * page + 1) for _ in range(n)]
            ok = s.reserve(gpu, rows, want)
            lens = list(s.book.lens)
            for r, w, y in zip(rows, want, ok):
                if y:
                    lens[r] = max(lens[r], w)
            s.set_lens(lens)
        elif what == "fork":
            s.fork(gpu, [rng.randrange(R) for _ in range(n)], [rng.randrange(R) for _ in range(n)])
        elif what == "free":
            s.free(gpu, [rng.randrange(R) for _ in range(n)])
        else:
            s.compact(gpu, in_place=rng.random() < 0.5)


@pytest.mark.gpu
def test_many_requests_and_a_large_pool(gpu):
    """More requests than a block has threads, more pages than one scan holds."""
    R, P = 3000, 70001
    s = Both(R, 8, P, 1, 2, 8, "latent", 7)
    s.reserve(gpu, list(range(0, R, 2)), [1 + (i * 7) % 16 for i in range(0, R, 2)])
    s.set_lens([1 + (i * 7) % 16 if i % 2 == 0 else 0 for i in range(R)])
    s.fork(gpu, list(range(0, R, 2)), list(range(1, R, 2)))
    s.free(gpu, list(range(0, R, 3)))
    s.compact(gpu)


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu):
    """A pool of more than 2^32 elements, forked from and compacted between its
    ends."""
    P, Hkv, page, d = 34000, 8, 128, 128
    k = torch.zeros((P, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(33)
    rows = torch.randn((2, Hkv, page, d), generator=g, device="cuda").bfloat16()
    k[P - 1], k[P - 2] = rows[0], rows[1]
    table, lens, refs = int32([[P - 1, P - 2, -1], [-1, -1, -1]]), int32([200, 0]), torch.zeros(P, dtype=torch.int32,
                                                                                             device="cuda")
    refs[P - 2:] = 1
    refs[: P - 4] = 1  # the lowest free page is far up
    fresh, ok = gpu.pages_fork(k, None, table, lens, refs, int32([0]), int32([1]))
    assert fresh.tolist() == [P - 4] and ok.tolist() == [1]
    assert torch.equal(k[P - 4, :, :72], rows[1][:, :72]) and not k[P - 4, :, 72:].any()
    assert table.tolist() == [[P - 1, P - 2, -1], [P - 1, P - 4, -1]] and refs[P - 1] == 2
    refs[: P - 4] = 0
    live = gpu.pages_compact(k, None, table, refs)
    assert live.tolist() == [3] and table.tolist() == [[2, 1, -1], [2, 0, -1]]
    assert refs[:4].tolist() == [1, 1, 2, 0] and int(refs.sum()) == 4
    assert torch.equal(k[2], rows[0]) and torch.equal(k[1], rows[1]) and torch.equal(k[0, :, :72], rows[1][:, :72])


@pytest.mark.gpu
@pytest.mark.parametrize("layout,Hkv,d", [("hnd", 2, 64), ("latent", 1, 576)])
def test_captured_and_replayed(gpu, layout, Hkv, d):
    """A whole round of upkeep in one graph, replayed on states it was not
    captured on, next to a second graph on its own state and stream."""
    page, P, R, width, n = 16, 300, 80, 8, 40

    def fresh_state(seed):
        s = Both(R, width, P, Hkv, page, d, layout, seed)
        rng = random.Random(seed)
        s.reserve(gpu, [0, 1, 2], [rng.randrange(1, 100) for _ in range(3)])
        s.set_lens([rng.randrange(1, 100) if r < 3 else 0 for r in range(R)])
        return s

    parents, children = [i % 3 for i in range(n)], list(range(3, 3 + n))
    want = [100 + i % 20 for i in range(n)]
    ids = [int32(x) for x in (parents, children, want, [4, 5, 0])]

    def round_of(s):
        fresh, ok = gpu.pages_fork(s.k, s.v, s.table, s.lens, s.refs, ids[0], ids[1])
        got = gpu.pages_reserve(s.table, s.refs, ids[1], ids[2], page)
        gpu.pages_free(s.table, s.lens, s.refs, ids[3])
        live = gpu.pages_compact(s.k, s.v, s.table, s.refs)
        return fresh, ok, got, live

    states = [fresh_state(seed) for seed in (41, 42)]
    saved = [[x.clone() for x in (s.table, s.lens, s.refs, *s.pools())] for s in states]
    round_of(fresh_state(43))
    torch.cuda.synchronize()
    graphs = []
    for s in states:
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = round_of(s)
        graphs.append((graph, stream, out))
    for s, old in zip(states, saved):
        for x, y in zip((s.table, s.lens, s.refs, *s.pools()), old):
            x.copy_(y)
    torch.cuda.synchronize()
    for graph, stream, _ in graphs:
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    for s, (_, _, (fresh, ok, got, live)) in zip(states, graphs):
        f, granted, copies = s.book.fork(parents, children)
        for a, b, m in copies:
            for x in s.want:
                as4(x)[b, :, :m] = as4(x)[a, :, :m]
        assert fresh.tolist() == f and ok.tolist() == granted
        assert got.tolist() == s.book.reserve(children, want)
        s.book.free([4, 5, 0])
        count, moves = s.book.compact()
        for a, b in moves:
            for x in s.want:
                x[b] = x[a]
        assert live.tolist() == [count]
        s.same()


# ------------------------------------------------------------------ compact

@pytest.mark.gpu
@pytest.mark.parametrize("P,live", [(1, 0), (1, 1), (7, 7), (64, 0), (5000, 2500), (5000, 1), (5000, 4999),
                                    (1025, 1024)])
def test_compact(gpu, P, live):
    for in_place in (True, False):
        s = Both(3, 50, P, 2, 4, 16, "hnd", 8)
        rng = random.Random(P + live)
        ids = rng.sample(range(P), live)
        for p in ids:
            s.refs[p] = s.book.refs[p] = rng.randrange(1, 5)
        cells = [rng.choice(ids) if ids and rng.random() < 0.8 else -1 for _ in range(150)]
        s.table.copy_(int32(cells).view(3, 50))
        s.book.table = [cells[:50], cells[50:100], cells[100:]]
        s.compact(gpu, in_place)


# -------------------------------------------------- all of them, as they are used

@pytest.mark.gpu
@pytest.mark.parametrize("form", ["paged", "latent"])
def test_a_serving_run(gpu, form):
    """Prompts are reserved, appended and attended to; beams are forked, given
    different tokens and attended to; some are freed, the pool is compacted, and
    attention gives the same bits as before."""
    d, Hkv, G, page, P, R, width = (576, 1, 16, 16, 200, 10, 20) if form == "latent" else (64, 2, 3, 16, 200, 10, 20)
    s = Both(R, width, P, Hkv, page, d, "latent" if form == "latent" else "hnd", 11)
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    rnd = lambda *sh: torch.randn(sh, generator=g, device="cuda").bfloat16()
    dv = 512 if form == "latent" else d
    prompt = [37, 128, 250]
    seqs = {r: [rnd(Hkv, n, d), rnd(Hkv, n, d)] for r, n in enumerate(prompt)}

    def append(rows, new):
        pos = s.lens[rows].contiguous()
        rows_t = s.table[rows].contiguous()
        gpu.pages_append(new[0], None if form == "latent" else new[1], s.k, s.v, rows_t, pos)
        s.lens[rows] += new[0].shape[2]

    def attend(rows, T, q):
        table, lens = s.table[rows].contiguous(), s.lens[rows].contiguous()
        if form == "latent":
            return gpu.attn_decode_latent(q, s.k, table, lens, 0.05)
        return gpu.attn_decode_paged(q, s.k, s.v, table, lens)

    def expect(rows, q):
        """The same attention over each sequence laid out as one page."""
        longest = max(seqs[r][0].shape[1] for r in rows)
        k, v = (torch.zeros((len(rows), Hkv, longest, x), dtype=torch.bfloat16, device="cuda") for x in (d, dv))
        for i, r in enumerate(rows):
            n = seqs[r][0].shape[1]
            k[i, :, :n] = seqs[r][0]
            v[i, :, :n] = seqs[r][0][..., :dv] if form == "latent" else seqs[r][1]
        table = torch.arange(len(rows), device="cuda").int().view(-1, 1)
        return attention(q, k, v, table, int32([seqs[r][0].shape[1] for r in rows]),
                         0.05 if form == "latent" else 1 / math.sqrt(d))

    assert gpu.pages_reserve(s.table, s.refs, int32([0, 1, 2]), int32([n + 1 for n in prompt]), page).tolist() == [1] * 3
    for r, n in enumerate(prompt):
        append([r], [x[None] for x in seqs[r]])
    q = rnd(3, Hkv * G, 1, d)
    check(*attend([0, 1, 2], 1, q), expect([0, 1, 2], q))
    # two beams of each prompt, two tokens each
    parents, children = [0, 0, 1, 1, 2, 2], [3, 4, 5, 6, 7, 8]
    _, ok = gpu.pages_fork(s.k, s.v, s.table, s.lens, s.refs, int32(parents), int32(children))
    assert ok.tolist() == [1] * 6
    assert gpu.pages_reserve(s.table, s.refs, int32(children), s.lens[children] + 2, page).tolist() == [1] * 6
    new = [rnd(6, Hkv, 2, d), rnd(6, Hkv, 2, d)]
    append(children, new)
    for i, (f, c) in enumerate(zip(parents, children)):
        seqs[c] = [torch.cat([x, y[i]], 1) for x, y in zip(seqs[f], new)]
    q = rnd(6, Hkv * G, 2, d)
    check(*attend(children, 2, q), expect(children, q))
    # the prompts and some beams go; the others keep their bits
    gpu.pages_free(s.table, s.lens, s.refs, int32([0, 1, 2, 4, 5]))
    left = [3, 6, 7, 8]
    q = rnd(4, Hkv * G, 1, d)
    before = attend(left, 1, q)
    check(*before, expect(left, q))
    live = int(gpu.pages_compact(s.k, s.v, s.table, s.refs))
    held = s.table[s.table >= 0]
    assert int(held.max()) < live and held.unique().numel() == live
    after = attend(left, 1, q)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert gpu.sync_status() == gpu.ATTN_OK
