"""The cache's page operations against a model of them in Python: books and page contents are equal."""
import random

import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """What the header says of each call, on lists."""

    def __init__(self, c):
        s = c.s
        self.pages, self.page, self.slots, self.width = s.pages, s.page_size, s.slots, s.width
        self.head, self.lens, self.refs = [0] * 4, [0] * s.slots, [0] * s.pages
        self.tables = [[-1] * s.width for _ in range(s.slots)]
        self.k, self.v = c.k.cpu().clone(), c.v.cpu().clone()
        self.where = []

    def need(self, n):
        return -(-n // self.page)

    def free_pages(self):
        return [p for p in range(self.pages) if self.refs[p] == 0]

    def extend(self, seqs, offsets):
        free, at, self.where = self.free_pages(), 0, [-1] * max(0, offsets[-1])
        for i, s in enumerate(seqs):
            a, b = offsets[i], offsets[i + 1]
            if not 0 <= s < self.slots or b < a:
                self.head[0] |= tfx.CACHE_BAD
                continue
            old, new = self.lens[s], self.lens[s] + b - a
            if self.need(new) > self.width:
                self.head[0] |= tfx.CACHE_TABLE_FULL
                continue
            more = self.need(new) - self.need(old)
            at += more
            if more and at > len(free):
                self.head[0] |= tfx.CACHE_FULL
                continue
            for j in range(more):
                p = free[at - more + j]
                self.tables[s][self.need(old) + j] = p
                self.refs[p] = 1
            self.lens[s] = new
            for t in range(a, b):
                pos = old + t - a
                self.where[t] = self.tables[s][pos // self.page] * self.page + pos % self.page

    def append(self, layer, k, v):
        for t in range(min(len(self.where), k.shape[0])):
            if self.where[t] >= 0:
                p, r = divmod(self.where[t], self.page)
                self.k[layer, p, r], self.v[layer, p, r] = k[t], v[t]

    def copy(self, src, dst):
        for a, b in zip(src, dst):
            if not (0 <= a < self.pages and 0 <= b < self.pages):
                self.head[0] |= tfx.CACHE_BAD
                continue
            self.k[:, b], self.v[:, b] = self.k[:, a].clone(), self.v[:, a].clone()

    def fork(self, src, dst):
        free, at = self.free_pages(), 0
        for s, d in zip(src, dst):
            if not (0 <= s < self.slots and 0 <= d < self.slots) or s == d or self.lens[d]:
                self.head[0] |= tfx.CACHE_BAD
                continue
            n, full = self.lens[s], self.lens[s] // self.page
            part = n % self.page != 0
            at += part
            if part and at > len(free):
                self.head[0] |= tfx.CACHE_FULL
                continue
            self.tables[d] = self.tables[s][:full] + [-1] * (self.width - full)
            for p in self.tables[s][:full]:
                self.refs[p] += 1
            if part:
                self.tables[d][full] = free[at - 1]
                self.refs[free[at - 1]] = 1
                self.copy([self.tables[s][full]], [free[at - 1]])
            self.lens[d] = n

    def free(self, seqs):
        for s in seqs:
            if not 0 <= s < self.slots:
                self.head[0] |= tfx.CACHE_BAD
                continue
            for j in range(self.need(self.lens[s])):
                self.refs[self.tables[s][j]] -= 1
                self.tables[s][j] = -1
            self.lens[s] = 0

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        free = [p for p in range(used) if self.refs[p] == 0]
        to = dict(zip([p for p in range(used, self.pages) if self.refs[p] > 0], free))
        for a, b in to.items():
            self.refs[a], self.refs[b] = 0, self.refs[a]
            self.copy([a], [b])
        self.tables = [[to.get(p, p) for p in row] for row in self.tables]
        self.head[1] = len(to)

    def agrees(self, c):
        book = self.head + self.lens + self.refs + [p for row in self.tables for p in row]
        assert c.book.tolist() == book
        assert torch.equal(c.k.cpu(), self.k) and torch.equal(c.v.cpu(), self.v)


def make(layers=2, pages=40, page=16, heads=2, dim=128, slots=12, width=9, dtype=torch.float16):
    k = torch.randn(layers, pages, page, heads, dim, device="cuda").to(dtype)
    c = tfx.Cache(k, torch.randn_like(k), slots, width)
    tfx.cache_reserve(c, slots, heads)
    return c, Model(c)


def rows_of(c, n):
    return (torch.randn(n, c.s.heads_kv, c.s.dim, device="cuda").to(c.k.dtype) for _ in range(2))


def grow(c, m, seqs, adds, layer=0):
    off = [0]
    for a in adds:
        off.append(off[-1] + a)
    tfx.cache_extend(c, dev(seqs), dev(off))
    m.extend(seqs, off)
    k, v = rows_of(c, off[-1])
    tfx.cache_append(c, layer, k, v, dev(seqs), dev(off))
    m.append(layer, k.cpu(), v.cpu())


@pytest.mark.parametrize("seed,page,heads,dim,dtype", [(0, 16, 2, 128, torch.float16), (1, 32, 1, 256, torch.bfloat16),
                                                       (2, 64, 3, 128, torch.float16), (3, 128, 1, 128, torch.bfloat16)])
def test_random_life(seed, page, heads, dim, dtype):
    """Sixty random steps; they run out of pages, slots and table room now and then."""
    rng = random.Random(seed)
    c, m = make(layers=2, pages=45, page=page, heads=heads, dim=dim, slots=12, width=9, dtype=dtype)
    for _ in range(60):
        op = rng.choice(["grow", "grow", "grow", "step", "fork", "free", "compact", "copy"])
        if op == "grow":
            seqs = rng.sample(range(12), rng.randint(1, 4))
            grow(c, m, seqs, [rng.choice([0, 1, page - 1, page, rng.randint(1, 4 * page)]) for _ in seqs], rng.randrange(2))
        elif op == "step":
            seqs = rng.sample(range(12), rng.randint(1, 12))
            grow(c, m, seqs, [1] * len(seqs), rng.randrange(2))
        elif op == "fork":
            some = rng.sample(range(12), 6)
            n = rng.randint(1, 3)
            src, dst = [rng.choice(some[3:]) for _ in range(n)], some[:n]
            tfx.cache_fork(c, dev(src), dev(dst))
            m.fork(src, dst)
        elif op == "free":
            seqs = rng.sample(range(12), rng.randint(1, 3))
            tfx.cache_free(c, dev(seqs))
            m.free(seqs)
        elif op == "compact":
            tfx.cache_compact(c)
            m.compact()
        else:
            some = rng.sample(range(45), 6)
            tfx.cache_copy(c, dev(some[:3]), dev(some[3:]))
            m.copy(some[:3], some[3:])
        m.agrees(c)


def test_fork_many_lengths_and_free_listed_twice():
    c, m = make(pages=64, slots=16, width=6)
    grow(c, m, list(range(6)), [0, 1, 15, 16, 17, 80])
    src, dst = [5, 4, 3, 2, 1, 0, 5, 4], [6, 7, 8, 9, 10, 11, 12, 13]
    tfx.cache_fork(c, dev(src), dev(dst))
    m.fork(src, dst)
    m.agrees(c)
    tfx.cache_free(c, dev([5, 6, 5, 4]))
    m.free([5, 6, 4])
    m.agrees(c)
    tfx.cache_compact(c)
    m.compact()
    m.agrees(c)
    assert c.status() == 0


def test_a_pool_larger_than_one_round_of_the_scan():
    """Free pages are looked for in rounds of 8192."""
    c, m = make(layers=1, pages=20011, page=16, heads=1, dim=128, slots=8, width=20011)
    grow(c, m, [0, 1], [16 * 8190, 16 * 9000])
    tfx.cache_free(c, dev([0]))
    m.free([0])
    grow(c, m, [2, 3], [16 * 8195, 33])
    m.agrees(c)
    tfx.cache_free(c, dev([1, 3]))
    m.free([1, 3])
    tfx.cache_compact(c)
    m.compact()
    m.agrees(c)


def test_refusals_on_the_device():
    """What only the device can see leaves its bit, and the rest as it was."""
    c, m = make(pages=6, slots=4, width=4)
    grow(c, m, [0, 9, -1, 1], [20, 3, 2, 16])
    m.agrees(c)
    assert c.status() == tfx.CACHE_BAD
    c.book[0] = m.head[0] = 0
    grow(c, m, [2, 3], [70, 16])
    m.agrees(c)
    assert c.status() == tfx.CACHE_TABLE_FULL
    c.book[0] = m.head[0] = 0
    grow(c, m, [2, 3, 0], [40, 1, 5])  # two pages are left: slot 2 finds too few, and slot 3 after it
    m.agrees(c)
    assert c.status() == tfx.CACHE_FULL
    c.book[0] = m.head[0] = 0
    for src, dst in (([0], [0]), ([0], [1]), ([5], [2]), ([0], [-3])):
        tfx.cache_fork(c, dev(src), dev(dst))
        m.fork(src, dst)
        m.agrees(c)
        assert c.status() == tfx.CACHE_BAD
        c.book[0] = m.head[0] = 0
    tfx.cache_copy(c, dev([0, 6, 1]), dev([5, 4, -1]))
    m.copy([0, 6, 1], [5, 4, -1])
    m.agrees(c)
    assert c.status() == tfx.CACHE_BAD
    tfx.cache_free(c, dev([7, 0]))
    m.free([7, 0])
    m.agrees(c)


def test_rows_past_the_offsets_are_not_stored():
    c, m = make()
    tfx.cache_extend(c, dev([3, 1]), dev([0, 5, 7]))
    m.extend([3, 1], [0, 5, 7])
    k, v = rows_of(c, 11)
    tfx.cache_append(c, 1, k, v)
    m.append(1, k.cpu(), v.cpu())
    m.agrees(c)


def test_append_of_pitched_rows():
    c, m = make()
    tfx.cache_extend(c, dev([0]), dev([0, 40]))
    m.extend([0], [0, 40])
    x = torch.randn(40, 2 * 256 + 8, device="cuda").half()
    k, v = x[:, :256].unflatten(1, (2, 128)), x[:, 256:512].unflatten(1, (2, 128))
    tfx.cache_append(c, 0, k, v)
    m.append(0, k.cpu(), v.cpu())
    m.agrees(c)
