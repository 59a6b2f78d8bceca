"""Upkeep of a paged cache's rows on the GPU against a plain model of the rules on the host: whole numbers and copies, equal."""
import random

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """The rules of gdn_cache_update and gdn_cache_compact, step by step."""

    def __init__(self, c):
        self.page = c.page_size
        self.table, self.lens, self.refs = c.table.tolist(), c.lens.tolist(), c.refs.tolist()
        self.pages, self.scales = c.pages.view(torch.uint8).clone(), c.scales.clone()
        self.W = c.table.shape[1]

    def used(self, r):
        return -(-self.lens[r] // self.page)

    def update(self, drop=(), fork=(), grow=None):
        R = len(self.lens)
        first = {}
        for a, b in fork:
            if 0 <= a < R and 0 <= b < R and a != b:
                first.setdefault(b, a)
        freed = {r for r in drop if 0 <= r < R} | set(first)
        for r in freed:
            for w in range(self.used(r)):
                self.refs[self.table[r][w]] -= 1
            self.lens[r] = 0
        for b, a in first.items():
            if a not in freed:
                self.table[b], self.lens[b] = list(self.table[a]), self.lens[a]
                for w in range(self.used(b)):
                    self.refs[self.table[b][w]] += 1
        if grow is None:
            return None
        free = [i for i, n in enumerate(self.refs) if n == 0]
        shared = [self.lens[r] % self.page > 0 and self.refs[self.table[r][self.used(r) - 1]] > 1 for r in range(R)]
        granted, place = [], 0
        for r, g in enumerate(grow):
            g = max(g, 0)
            if self.lens[r] + g > self.W * self.page:
                granted.append(-1)
                continue
            have, copy = self.used(r), g > 0 and shared[r]
            need = -(-(self.lens[r] + g) // self.page) - have + copy
            mine, place = free[place:place + need], place + need
            if need and place > len(free):
                granted.append(-1)
                continue
            if copy:
                old, new = self.table[r][have - 1], mine.pop(0)
                self.refs[old] -= 1
                self.table[r][have - 1] = new
                self.pages[:, new], self.scales[:, new] = self.pages[:, old], self.scales[:, old]
                self.refs[new] = 1
            for w, pg in enumerate(mine):
                self.table[r][have + w] = pg
                self.refs[pg] = 1
            self.lens[r] += g
            granted.append(g)
        return granted

    def compact(self):
        n = sum(x > 0 for x in self.refs)
        movers = [i for i, x in enumerate(self.refs) if x > 0 and i >= n]
        holes = [i for i, x in enumerate(self.refs) if x == 0 and i < n]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.pages[:, b], self.scales[:, b] = self.pages[:, a], self.scales[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for r in range(len(self.lens)):
            for w in range(self.used(r)):
                self.table[r][w] = to.get(self.table[r][w], self.table[r][w])
        return n

    def check(self, c):
        torch.cuda.synchronize()
        assert gdn.read_status("cuda") == gdn.GDN_OK
        assert c.lens.tolist() == self.lens and c.refs.tolist() == self.refs
        got = c.table.tolist()
        for r in range(len(self.lens)):
            assert got[r][:self.used(r)] == self.table[r][:self.used(r)], r
        # what rows hold; freed pages may keep anything
        held = torch.tensor([i for i, n in enumerate(self.refs) if n > 0], dtype=torch.long, device="cuda")
        assert torch.equal(c.pages.view(torch.uint8)[:, held], self.pages[:, held])
        assert torch.equal(c.scales[:, held], self.scales[:, held])


def fresh(R=6, N=40, W=8, page=16, H=1, D=32, L=2, seed=0):
    c = gdn.PagedCache.empty(L, N, H, D, R, W, page_size=page)
    g = torch.Generator(device="cuda").manual_seed(seed)
    c.pages.view(torch.uint8).copy_(torch.randint(0, 127, c.pages.shape, generator=g, device="cuda", dtype=torch.uint8))
    c.scales.copy_(torch.rand(c.scales.shape, generator=g, device="cuda"))
    return c


def step(c, m, drop=None, fork=None, grow=None):
    granted = gdn.gdn_cache_update(c, drop=None if drop is None else ints(*drop),
                                   fork_from=None if fork is None else ints(*[a for a, _ in fork]),
                                   fork_to=None if fork is None else ints(*[b for _, b in fork]),
                                   grow=None if grow is None else ints(*grow))
    want = m.update(drop or (), fork or (), grow)
    assert granted is None if want is None else granted.tolist() == want
    m.check(c)


@pytest.mark.parametrize("page, H, D, L", [(16, 1, 32, 1), (64, 3, 64, 2), (128, 8, 128, 3)])
def test_a_few_turns(page, H, D, L):
    """A prefix, forks of it, growth with copies of the shared page (the last holder has its own), freeing, compaction."""
    c = fresh(page=page, H=H, D=D, L=L)
    m = Model(c)
    p = page
    step(c, m, grow=[2 * p + 5, 0, 0, 0, 0, 0])
    step(c, m, fork=[(0, 1), (0, 3), (0, 5)])
    step(c, m, grow=[0, 1, 0, p, 0, 0])
    step(c, m, grow=[1, 1, 1, 1, 1, 1])          # row 0 and row 5 share their last page: both copy it
    step(c, m, drop=[1], fork=[(3, 2), (0, 4)], grow=[0, 7, 3, 0, 0, 2 * p])
    assert int(gdn.gdn_cache_compact(c)) == m.compact()
    m.check(c)
    step(c, m, drop=[0, 1, 2, 3, 4])
    assert int(gdn.gdn_cache_compact(c)) == m.compact()
    m.check(c)
    assert int(gdn.gdn_cache_compact(c)) == m.compact()
    m.check(c)


def test_whole_shared_pages_are_not_copied():
    c = fresh()
    m = Model(c)
    step(c, m, grow=[32, 0, 0, 0, 0, 0])
    step(c, m, fork=[(0, 1), (0, 2)], grow=[0, 1, 17, 0, 0, 0])
    assert m.refs.count(3) == 2


def test_odd_lists():
    """The same row twice, rows that do not exist, forks of themselves, of rows just freed and of rows forked at the same
    time, two forks of one row: freed once, the first pair counts, a freed source leaves an empty row."""
    c = fresh()
    m = Model(c)
    step(c, m, grow=[20, 40, 5, 0, 33, 16])
    step(c, m, drop=[2, 2, -1, 6, 2 ** 31 - 1, -2 ** 31, 2])
    step(c, m, fork=[(0, 3), (1, 3), (0, 0), (9, 1), (1, -1), (4, 2), (4, 2)])
    step(c, m, drop=[0], fork=[(0, 1), (4, 5), (5, 2)])   # 0 is freed, 5 is a destination
    assert m.lens[1] == 0 and m.lens[2] == 0 and m.lens[5] == 33
    step(c, m, drop=[], fork=[], grow=[0] * 6)
    step(c, m, grow=[-5, 3, -2 ** 31, 0, 0, 0])


def test_too_few_pages():
    """Rows are served in order until one finds too few pages; those after it that need none are served still."""
    c = fresh(N=10)
    m = Model(c)
    step(c, m, grow=[40, 16, 10, 0, 90, 1])       # 3 + 1 + 1 pages; 6 where 5 are left; then 1
    assert m.lens == [40, 16, 10, 0, 0, 0]
    step(c, m, grow=[8, 0, 6, 128, 129, 0])       # room in the last pages; too many; past the table's width
    step(c, m, grow=[0, 0, 0, 2 ** 31 - 1, 0, 80])


def test_every_page_taken_and_none_free():
    c = fresh(N=6, W=6)
    m = Model(c)
    step(c, m, grow=[96, 0, 0, 0, 0, 0])
    step(c, m, grow=[0, 1, 0, 0, 0, 0])
    step(c, m, fork=[(0, 1)], grow=[0] * 6)
    step(c, m, drop=[0, 1])
    assert int(gdn.gdn_cache_compact(c)) == 0


@pytest.mark.parametrize("seed", range(6))
def test_random_turns(seed):
    r = random.Random(seed)
    R, N = r.choice([(5, 30), (40, 200), (1100, 3000), (70, 20001)])
    c = fresh(R=R, N=N, W=r.choice([3, 9]), page=16, L=r.choice([1, 2]), seed=seed)
    m = Model(c)
    for _ in range(12):
        some = lambda n: [r.randrange(-1, R + 1) for _ in range(r.randrange(n))]   # noqa: E731
        fork = list(zip(some(R // 2 + 2), some(R // 2 + 2)))
        step(c, m, drop=some(R // 2 + 2) if r.random() < 0.7 else None, fork=fork if r.random() < 0.7 else None,
             grow=[r.choice([0, 0, 1, 5, 16, 40, -1]) for _ in range(R)] if r.random() < 0.8 else None)
        if r.random() < 0.4:
            assert int(gdn.gdn_cache_compact(c)) == m.compact()
            m.check(c)


def test_many_rows():
    """The largest number of rows, more pages than one round of the scan looks through."""
    R = 16384
    c = fresh(R=R, N=3 * R, W=2, L=1)
    m = Model(c)
    step(c, m, grow=[1 + i % 32 for i in range(R)])
    step(c, m, drop=list(range(0, R, 2)))
    assert int(gdn.gdn_cache_compact(c)) == m.compact()
    m.check(c)
    step(c, m, fork=[(i + 1, i) for i in range(0, R, 2)], grow=[i % 2 for i in range(R)])


def test_pages_past_32_bits():
    """Copies behind the first 2^32 bytes of a layer, and in a layer behind the first."""
    c = gdn.PagedCache.empty(2, 9000, 8, 128, 3, 4, page_size=128)   # 2.4 GB a layer
    c.table[0, 0], c.lens[0] = 8999, 100
    c.refs.fill_(1)
    c.refs[8998] = 0
    c.refs[0] = 0
    c.pages.view(torch.uint8)[:, 8999] = 0x35
    c.scales[:, 8999] = 0.5
    gdn.gdn_cache_update(c, fork_from=ints(0), fork_to=ints(1), grow=ints(0, 1, 0))
    assert int(c.table[1, 0]) == 0 and (c.pages.view(torch.uint8)[:, 0] == 0x35).all() and (c.scales[:, 0] == 0.5).all()
    c.refs[100] = 0
    assert int(gdn.gdn_cache_compact(c)) == 8998
    assert int(c.table[0, 0]) in (100, 8998) and (c.pages.view(torch.uint8)[:, int(c.table[0, 0])] == 0x35).all()


def test_bad_pages_are_reported():
    for bad in (-1, 40, 2 ** 31 - 1):
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        c = fresh()
        gdn.gdn_cache_update(c, grow=ints(40, 20, 0, 0, 0, 0), ws=ws)
        assert gdn.read_status(ws=ws) == gdn.GDN_OK
        refs = c.refs.tolist()
        c.table[0, 1] = bad
        gdn.gdn_cache_compact(c, ws=ws)
        assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
        gdn.clear_status(ws=ws)
        gdn.gdn_cache_update(c, drop=ints(0), ws=ws)
        assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
        assert sum(refs) - c.refs.sum().item() == 2 and c.lens.tolist()[:2] == [0, 20]


def test_captured():
    """A captured turn follows its lists: growth by one token a row, page after page."""
    c = fresh(N=60, W=9)
    m = Model(c)
    grow, src, dst = ints(1, 1, 1, 0, 0, 0), ints(0), ints(-1)
    gdn.gdn_cache_update(c, grow=ints(9, 15, 16, 0, 0, 0))
    m.update(grow=[9, 15, 16, 0, 0, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        granted = gdn.gdn_cache_update(c, fork_from=src, fork_to=dst, grow=grow)
        live = gdn.gdn_cache_compact(c)
    for i in range(20):
        to = 3 + i % 3 if i % 4 == 0 else -1
        dst.fill_(to)
        graph.replay()
        assert granted.tolist() == m.update(fork=[(0, to)], grow=[1, 1, 1, 0, 0, 0])
        assert int(live) == m.compact()
        m.check(c)
