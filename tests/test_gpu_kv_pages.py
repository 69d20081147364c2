"""The paged cache's upkeep against a model of it in Python: every number and every byte equal."""
import random

import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tests.helpers import requires_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    requires_gpu()


class Cache:
    """The library's cache and its model, changed side by side."""

    def __init__(self, pages, seqs, wide, page, npools=2, width=8, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.page, self.wide = page, wide
        self.pools = [torch.randn(pages, page, width, generator=g, device="cuda").to(dtype) for _ in range(npools)]
        self.m_pools = [p.clone() for p in self.pools]
        ints = dict(device="cuda", dtype=torch.int32)
        self.refs, self.lens = torch.zeros(pages, **ints), torch.zeros(seqs, **ints)
        self.store = torch.full((seqs, wide + 2), -5, **ints)
        self.table = self.store[:, :wide]
        self.table.fill_(-1)
        self.m_refs, self.m_lens, self.m_table = [0] * pages, [0] * seqs, [[-1] * wide for _ in range(seqs)]

    def ints(self, v):
        return torch.tensor(v, device="cuda", dtype=torch.int32)

    def same(self):
        assert self.refs.tolist() == self.m_refs and self.lens.tolist() == self.m_lens
        assert self.table.tolist() == self.m_table
        assert bool((self.store[:, self.wide:] == -5).all())
        for a, b in zip(self.pools, self.m_pools):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))

    def count(self, n):
        return -(-n // self.page)

    def take(self, asks):
        """asks: [(entry, pages)] of those that can be; the entries that get theirs and which."""
        free, got, upto = [p for p, r in enumerate(self.m_refs) if r == 0], {}, 0
        for e, n in asks:
            upto += n
            if upto <= len(free):
                got[e] = free[upto - n:upto]
        return got

    def reserve(self, seqs, add):
        ok = self.ints([-1] * len(seqs))
        tgc.tgc_kv_reserve(self.refs, self.table, self.lens, self.ints(seqs), self.ints(add), self.page, ok=ok)
        asks, seen = [], set()
        for e, (s, n) in enumerate(zip(seqs, add)):
            if 0 <= s < len(self.m_lens) and s not in seen:
                seen.add(s)
                if n >= 0 and self.m_lens[s] + n <= self.wide * self.page:
                    asks.append((e, self.count(self.m_lens[s] + n) - self.count(self.m_lens[s])))
        got = self.take(asks)
        for e, pages in got.items():
            s = seqs[e]
            have = self.count(self.m_lens[s])
            for i, p in enumerate(pages):
                self.m_table[s][have + i], self.m_refs[p] = p, 1
            self.m_lens[s] += add[e]
        assert ok.tolist() == [int(e in got) for e in range(len(seqs))]

    def fork(self, src, dst):
        ok = self.ints([-1] * len(src))
        tgc.tgc_kv_fork(self.pools, self.refs, self.table, self.lens, self.ints(src), self.ints(dst), self.page, ok=ok)
        asks, seen, S = [], set(), len(self.m_lens)
        for e, (a, b) in enumerate(zip(src, dst)):
            if not 0 <= b < S or b in seen:
                continue
            seen.add(b)
            if 0 <= a < S and a != b and self.m_lens[b] == 0:
                asks.append((e, int(self.m_lens[a] % self.page > 0)))
        got, lens = self.take(asks), list(self.m_lens)
        for e, pages in got.items():
            a, b = src[e], dst[e]
            whole = lens[a] // self.page
            for i in range(whole):
                self.m_table[b][i] = self.m_table[a][i]
                self.m_refs[self.m_table[a][i]] += 1
            for p in pages:
                self.m_table[b][whole], self.m_refs[p] = p, 1
                for pool in self.m_pools:
                    pool[p] = pool[self.m_table[a][whole]]
            self.m_lens[b] = lens[a]
        assert ok.tolist() == [int(e in got) for e in range(len(src))]

    def free(self, seqs):
        tgc.tgc_kv_free(self.refs, self.table, self.lens, self.ints(seqs))
        for s in seqs:
            if 0 <= s < len(self.m_lens):
                for p in self.m_table[s]:
                    if p >= 0:
                        self.m_refs[p] -= 1
                self.m_table[s], self.m_lens[s] = [-1] * self.wide, 0

    def compact(self):
        used = self.ints([-1])
        tgc.tgc_kv_compact(self.pools, self.refs, self.table, used)
        n = sum(r > 0 for r in self.m_refs)
        movers = [p for p in range(n, len(self.m_refs)) if self.m_refs[p] > 0]
        to = dict(zip(movers, [p for p in range(n) if self.m_refs[p] == 0]))
        for a, b in to.items():
            self.m_refs[b], self.m_refs[a] = self.m_refs[a], 0
            for pool in self.m_pools:
                pool[b] = pool[a]
        self.m_table = [[to.get(p, p) for p in row] for row in self.m_table]
        assert used.tolist() == [n]


@pytest.mark.parametrize("pages,seqs,wide,page,npools,width", [
    (40, 12, 6, 4, 2, 8), (100, 30, 10, 1, 1, 8), (5000, 60, 200, 16, 3, 24), (2048, 40, 90, 7, 2, 16), (2049, 40, 90, 3, 4, 40),
    (7, 5, 3, 100, 2, 8), (300, 1500, 4, 2, 2, 8), (9000, 8, 3000, 2, 1, 8)])
def test_random_histories(pages, seqs, wide, page, npools, width):
    """Reserves, forks, frees and compactions at random, bad and repeated entries among them, pages running out."""
    c, rng = Cache(pages, seqs, wide, page, npools, width, seed=pages), random.Random(pages)
    some = lambda n: [rng.choice([rng.randrange(seqs)] * 12 + [-1, seqs, 2 ** 31 - 1]) for _ in range(n)]  # noqa: E731
    for _ in range(25):
        n = rng.choice([1, 2, seqs // 3 + 1, seqs])
        kind = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        if kind == "reserve":
            most = max(1, pages * page // seqs)
            c.reserve(some(n), [rng.choice([0, 1, 1, rng.randrange(3 * most), -1, wide * page + 1]) for _ in range(n)])
        elif kind == "fork":
            c.fork(some(n), some(n))
        elif kind == "free":
            c.free(some(n // 2 + 1))
        else:
            c.compact()
        c.same()


def test_many_pages_and_entries():
    c = Cache(200000, 3000, 300, 2, 1, 8, seed=1)
    rng = random.Random(1)
    c.reserve(list(range(2000)), [rng.randrange(150) for _ in range(2000)])
    c.free(rng.sample(range(2000), 700))
    c.fork([rng.randrange(2000) for _ in range(900)], list(range(2050, 2950)))
    c.same()
    c.compact()
    c.same()
    c.compact()  # nothing left to move
    c.same()


@pytest.mark.parametrize("n", [4, 1100])
def test_the_most_pages(n):
    """2^31 - 4096 pages, all but four of them taken: those are found, at the start and the end, and the entry that
    wants more makes the search run to the pool's very end."""
    pages = 2 ** 31 - 4096
    ints = dict(device="cuda", dtype=torch.int32)
    refs, table, lens = torch.ones(pages, **ints), torch.full((4, 4), -1, **ints), torch.zeros(4, **ints)
    refs[5] = 0
    refs[-3:] = 0
    seqs, add = torch.full((n,), -1, **ints), torch.zeros(n, **ints)
    seqs[:3], add[:3], ok = torch.tensor([0, 1, 2], **ints), torch.tensor([2, 2, 1], **ints), torch.full((n,), -1, **ints)
    tgc.tgc_kv_reserve(refs, table, lens, seqs, add, 1, ok=ok)
    assert table[:, :2].tolist() == [[5, pages - 3], [pages - 2, pages - 1], [-1, -1], [-1, -1]]
    assert ok.tolist() == [1, 1] + [0] * (n - 2) and lens.tolist() == [2, 2, 0, 0]
    assert bool((refs == 1).all())


@pytest.mark.parametrize("page_bytes", [16, 48, 512, 4096, 4112, 40960])
@pytest.mark.parametrize("npools", [1, 5, 256])
def test_copy(page_bytes, npools):
    g = torch.Generator(device="cuda").manual_seed(page_bytes)
    a = [torch.randint(0, 256, (30, page_bytes), generator=g, device="cuda", dtype=torch.uint8) for _ in range(npools)]
    b = [torch.randint(0, 256, (20, page_bytes), generator=g, device="cuda", dtype=torch.uint8) for _ in range(npools)]
    src = torch.tensor([3, 29, 0, 3, -1, 30, 5], device="cuda", dtype=torch.int32)
    dst = torch.tensor([19, 0, 7, 8, 9, 10, 20], device="cuda", dtype=torch.int32)
    want = [t.clone() for t in b]
    for x, w in zip(a, want):
        for i, j in ((3, 19), (29, 0), (0, 7), (3, 8)):
            w[j] = x[i]
    tgc.tgc_kv_copy(b, a, dst, src)
    assert all(torch.equal(x, w) for x, w in zip(b, want))
    tgc.tgc_kv_copy(b, b, dst[:1], src[:1])  # inside one cache: page 3 to 19
    assert all(torch.equal(x[19], x[3]) for x in b)


def test_corrupt_bookkeeping_stays_inside():
    """Table entries, lengths and references that no history gives: no access outside (the bytes around stay), no claim
    about what the cache holds then."""
    ints = dict(device="cuda", dtype=torch.int32)
    wall = torch.full((3, 64), 77, **ints)  # refs, table rows, lens each between two walls
    refs, table, lens = wall[0, 16:48], wall[1, 16:48].view(4, 8), wall[2, 16:20]
    pool = torch.zeros(34, 4, 8, device="cuda", dtype=torch.bfloat16)
    refs.copy_(torch.arange(32) % 5 - 2)
    table.copy_(torch.tensor([[2 ** 31 - 1, -(2 ** 31), 31, 32] * 2] * 4))
    lens.copy_(torch.tensor([2 ** 31 - 1, -9, 30, 0]))
    seqs = torch.tensor([0, 1, 2, 3, 3, -1, 4], **ints)
    tgc.tgc_kv_reserve(refs, table, lens, seqs, torch.full_like(seqs, 5), 4)
    tgc.tgc_kv_fork([pool[1:33]], refs, table, lens, torch.tensor([0, 2, 1], **ints), torch.tensor([3, 1, 0], **ints), 4)
    tgc.tgc_kv_compact([pool[1:33]], refs, table)
    tgc.tgc_kv_free(refs, table, lens, seqs)
    torch.cuda.synchronize()
    assert bool((wall[:, :16] == 77).all()) and bool((wall[:2, 48:] == 77).all()) and bool((wall[2, 20:] == 77).all())
    assert not bool(pool.any())


def test_streams_and_graphs():
    c = Cache(64, 6, 8, 4, seed=3)
    c.reserve([0, 1], [13, 9])
    ok = c.ints([0, 0])
    seqs, add = c.ints([0, 1]), c.ints([1, 1])
    ws = torch.empty(tgc.tgc_kv_reserve_workspace_bytes(c.refs, c.table, c.lens, seqs, add, 4), device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tgc.tgc_kv_reserve(c.refs, c.table, c.lens, seqs, c.ints([0, 0]), 4, workspace=ws, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tgc.tgc_kv_reserve(c.refs, c.table, c.lens, seqs, add, 4, ok=ok, workspace=ws)
    for _ in range(5):
        graph.replay()
    assert c.lens.tolist()[:2] == [18, 14] and ok.tolist() == [1, 1]
    assert int((c.table >= 0).sum()) == 5 + 4 and int(c.refs.sum()) == 9


def test_every_call_on_another_stream_and_captured():
    """Reserve, free, fork, compact and a copy: the same on the current stream, on another one and replayed, each time
    from the same cache, and the model's."""
    caches = [Cache(600, 40, 20, 4, npools=3, width=16, seed=4) for _ in range(3)]
    rng = random.Random(4)
    adds, gone = [rng.randrange(60) for _ in range(40)], rng.sample(range(40), 15)
    add2 = [rng.randrange(9) for _ in range(40)]
    lists = {k: caches[0].ints(v) for k, v in dict(seqs=list(range(40)), adds=adds, gone=gone, src=[s for s in range(40) if s not in gone][:15],
                                                  add2=add2, a=[0, 1, 2], b=[597, 598, 599]).items()}
    side = torch.cuda.Stream()

    def work(c, **on):
        own = (lambda n: dict(workspace=torch.empty(n, device="cuda", dtype=torch.uint8))) if on.pop("captured", False) else (lambda n: {})
        grow = (c.refs, c.table, c.lens, lists["seqs"], lists["adds"], 4)
        tgc.tgc_kv_reserve(*grow, **on, **own(1 << 20))
        tgc.tgc_kv_free(c.refs, c.table, c.lens, lists["gone"], **on)
        tgc.tgc_kv_fork(c.pools, c.refs, c.table, c.lens, lists["src"], lists["gone"], 4, **on, **own(1 << 20))
        tgc.tgc_kv_reserve(c.refs, c.table, c.lens, lists["seqs"], lists["add2"], 4, **on, **own(1 << 20))
        tgc.tgc_kv_compact(c.pools, c.refs, c.table, **on, **own(1 << 20))
        tgc.tgc_kv_copy(c.pools, c.pools, lists["b"], lists["a"], **on)

    work(caches[0])
    torch.cuda.synchronize()
    work(caches[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(caches[2], captured=True)
    graph.replay()
    torch.cuda.synchronize()
    c = caches[0]
    for o in caches[1:]:
        assert torch.equal(c.refs, o.refs) and torch.equal(c.table, o.table) and torch.equal(c.lens, o.lens)
        assert all(torch.equal(x, y) for x, y in zip(c.pools, o.pools))
    m = Cache(600, 40, 20, 4, npools=3, width=16, seed=4)
    m.reserve(list(range(40)), adds)
    m.free(gone)
    m.fork([s for s in range(40) if s not in gone][:15], gone)
    m.reserve(list(range(40)), add2)
    m.compact()
    m.same()
    assert torch.equal(m.table, c.table) and torch.equal(m.lens, c.lens) and torch.equal(m.refs, c.refs)


def test_the_binding_refuses():
    c = Cache(8, 3, 4, 4)
    one = c.ints([0])
    for call in (lambda: tgc.tgc_kv_copy(c.pools, c.pools[:1], one, one), lambda: tgc.tgc_kv_copy([], [], one, one),
                 lambda: tgc.tgc_kv_copy(c.pools, [c.pools[0], c.pools[0][:4]], one, one), lambda: tgc.tgc_kv_copy(c.pools, c.pools, one, one.long()),
                 lambda: tgc.tgc_kv_copy([p[:, ::2] for p in c.pools], c.pools, one, one), lambda: tgc.tgc_kv_copy(c.pools, c.pools, one, c.ints([0, 1])),
                 lambda: tgc.tgc_kv_reserve(c.refs, c.table, c.lens[:2], one, one, 4), lambda: tgc.tgc_kv_reserve(c.refs, c.table, c.lens, one, one, 0),
                 lambda: tgc.tgc_kv_fork(c.pools, c.refs[:7], c.table, c.lens, one, one, 4), lambda: tgc.tgc_kv_fork(c.pools, c.refs, c.table, c.lens, one, one, 5),
                 lambda: tgc.tgc_kv_free(c.refs.float(), c.table, c.lens, one), lambda: tgc.tgc_kv_compact(c.pools, c.refs, c.table, c.ints([0, 0]))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(tgc.TGCError):
        tgc.tgc_kv_reserve(c.refs, c.table, c.lens, one, one, 4, workspace=torch.zeros(8, device="cuda", dtype=torch.uint8))
