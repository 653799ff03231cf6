"""Appends that do not directly follow their extend, against a model that keeps (slot, position) of every row."""
import random

import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx
from test_gpu_cache import Model, dev, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Rows(Model):
    """Where a list's rows go: the last tokens that each of its sequences has."""

    def put(self, layer, k, v, seqs, offsets):
        for s, a, b in zip(seqs, offsets, offsets[1:]):
            for t in range(a, b):
                p, r = divmod(self.lens[s] - (b - t), self.page)
                self.k[layer, self.tables[s][p], r], self.v[layer, self.tables[s][p], r] = k[t], v[t]


def make(layers=2, pages=40, page=16, heads=2, dim=128, slots=12, width=9):
    k = torch.randn(layers, pages, page, heads, dim, device="cuda").half()
    c = tfx.Cache(k, torch.randn_like(k), slots, width)
    tfx.cache_reserve(c, min(slots, 4096), heads)
    return c, Rows(c)


def extend(c, m, seqs, offsets):
    tfx.cache_extend(c, dev(seqs), dev(offsets))
    m.extend(seqs, offsets)


def append(c, m, seqs, offsets, listed, layers=(0, 1)):
    """All layers' rows of one extend; the lists left out where it was the last one."""
    for layer in layers:
        k, v = rows_of(c, offsets[-1])
        if listed:
            tfx.cache_append(c, layer, k, v, dev(seqs), dev(offsets))
        else:
            tfx.cache_append(c, layer, k, v)
        m.put(layer, k.cpu(), v.cpu(), seqs, offsets)
        m.agrees(c)


def filled():
    """Slots 0 to 3 hold 20, 33, 16 and 5 tokens, and slot 4 has gone and left free pages in between."""
    c, m = make()
    seqs, off = [0, 4, 1, 2, 3], [0, 20, 60, 93, 109, 114]
    extend(c, m, seqs, off)
    append(c, m, seqs, off, True)
    tfx.cache_free(c, dev([4]))
    m.free([4])
    return c, m


@pytest.mark.parametrize("listed", [False, True])
def test_fork_of_others_between(listed):
    c, m = filled()
    extend(c, m, [3, 1], [0, 30, 47])
    tfx.cache_fork(c, dev([0, 2]), dev([7, 8]))
    m.fork([0, 2], [7, 8])
    append(c, m, [3, 1], [0, 30, 47], listed)
    assert c.status() == 0


@pytest.mark.parametrize("listed", [False, True])
def test_compact_between(listed):
    """Pages have other numbers when the rows arrive; a compact that moves none stops nothing either."""
    c, m = filled()
    extend(c, m, [3, 1], [0, 30, 47])
    tfx.cache_free(c, dev([0]))
    m.free([0])
    tfx.cache_compact(c)
    m.compact()
    assert m.head[1] > 0
    append(c, m, [3, 1], [0, 30, 47], listed, (0,))
    tfx.cache_compact(c)
    m.compact()
    assert m.head[1] == 0
    append(c, m, [3, 1], [0, 30, 47], listed, (1,))
    assert c.status() == 0


def test_lists_of_an_extend_before_the_last():
    """A prefill step's list and a decode step's, extended one after the other, then layer by layer."""
    c, m = filled()
    a, aoff, b, boff = [5, 6], [0, 40, 57], [0, 1, 2, 3], [0, 1, 2, 3, 4]
    extend(c, m, a, aoff)
    extend(c, m, b, boff)
    for layer in (0, 1):
        append(c, m, a, aoff, True, (layer,))
        append(c, m, b, boff, layer == 0, (layer,))
    append(c, m, [6], [0, 17], True)  # a list's entries one at a time
    assert c.status() == 0


def test_a_slot_without_new_tokens_keeps_its_room():
    c, m = filled()
    extend(c, m, [3, 1], [0, 30, 47])
    extend(c, m, [0, 3, 2], [0, 4, 4, 6])
    append(c, m, [3, 1], [0, 30, 47], True)
    append(c, m, [0, 3, 2], [0, 4, 4, 6], False)
    assert c.status() == 0


@pytest.mark.parametrize("listed", [False, True])
def test_rows_of_a_freed_slot_are_not_stored(listed):
    """Its pages may be another's by then: here a fork's into the same slot."""
    c, m = filled()
    extend(c, m, [3, 1], [0, 30, 47])
    tfx.cache_free(c, dev([3]))
    m.free([3])
    tfx.cache_fork(c, dev([0]), dev([3]))
    m.fork([0], [3])
    k, v = rows_of(c, 47)
    tfx.cache_append(c, 0, k, v, *((dev([3, 1]), dev([0, 30, 47])) if listed else ()))
    m.put(0, k.cpu()[30:], v.cpu()[30:], [1], [0, 17])
    m.head[0] |= tfx.CACHE_BAD
    m.agrees(c)


def test_append_before_any_extend_stores_nothing():
    c, m = make()
    k, v = rows_of(c, 30)
    tfx.cache_append(c, 0, k, v)
    m.agrees(c)
    tfx.cache_append(c, 0, k, v, dev([1, 2]), dev([0, 10, 30]))
    m.head[0] |= tfx.CACHE_BAD
    m.agrees(c)


def test_lists_that_no_extend_had():
    """Another number of tokens, slots out of range, rows outside the list: not stored, each wrong entry flagged."""
    c, m = filled()
    extend(c, m, [3, 1], [0, 30, 47])
    k, v = rows_of(c, 60)
    tfx.cache_append(c, 0, k, v, dev([3, 1]), dev([5, 36, 53]))  # 31 tokens for slot 3
    m.put(0, k.cpu()[36:], v.cpu()[36:], [1], [0, 17])
    m.head[0] |= tfx.CACHE_BAD
    m.agrees(c)
    c.book[0] = m.head[0] = 0
    tfx.cache_append(c, 1, k, v, dev([1]), dev([9, 26]))  # right, nine rows late
    m.put(1, k.cpu()[9:], v.cpu()[9:], [1], [0, 17])
    m.agrees(c)
    for s in (-1, 12, 1 << 30):
        tfx.cache_append(c, 1, k, v, dev([s]), dev([0, 17]))
        m.head[0] |= tfx.CACHE_BAD
        m.agrees(c)
        c.book[0] = m.head[0] = 0


def test_rows_that_an_extend_refused():
    c, m = filled()
    extend(c, m, [3, 1, 9], [0, 150, 167, 167 + 145])  # slot 3 would need ten pages of its nine, slot 9 as many
    assert m.head[0] == tfx.CACHE_TABLE_FULL
    k, v = rows_of(c, 312)
    tfx.cache_append(c, 0, k, v)
    m.put(0, k.cpu()[150:], v.cpu()[150:], [1], [0, 17])
    m.agrees(c)


def test_compact_of_a_book_with_a_count_below_zero():
    """A caller's broken count: the page is free, and one that is moved there brings its own."""
    c, m = filled()
    tfx.cache_free(c, dev([0, 1]))
    m.free([0, 1])
    assert m.refs[:10] == [0] * 8 + [1, 1]
    c.refs[0] = -3
    tfx.cache_compact(c)
    m.compact()
    assert m.head[1] == 2
    m.agrees(c)


def test_lists_of_more_than_one_round():
    """Books are worked out 1024 entries at a time: growth, appends, forks and pages that run out in a later round."""
    n = 2500
    c, m = make(layers=1, pages=4200, page=16, heads=1, slots=2 * n, width=4)
    seqs = list(range(n))
    random.Random(1).shuffle(seqs)
    off = [0]
    for i in range(n):
        off.append(off[-1] + (i * 7) % 20)
    extend(c, m, seqs, off)
    assert c.status() == 0
    append(c, m, seqs, off, True, (0,))
    append(c, m, seqs, off, False, (0,))
    tfx.cache_fork(c, dev(seqs), dev([s + n for s in seqs]))
    m.fork(seqs, [s + n for s in seqs])
    m.agrees(c)
    assert c.status() == tfx.CACHE_FULL and any(m.lens[n:]) and not all(m.lens[n:])
    c.book[0] = m.head[0] = 0
    gone = [s for s in range(2 * n) if s % 3]
    tfx.cache_free(c, dev(gone))
    m.free(gone)
    tfx.cache_compact(c)
    m.compact()
    m.agrees(c)
    step = list(range(0, 2 * n, 2))
    extend(c, m, step, list(range(n + 1)))
    m.agrees(c)
    append(c, m, step, list(range(n + 1)), True, (0,))
    assert c.status() == 0


@pytest.mark.parametrize("n", [1, 31, 32, 33, 700, 1024, 1025])
def test_rows_find_their_entry(n):
    """Lists with empty entries at their ends and in between."""
    adds = [(0, 0, 3, 1, 0, 17)[(i * i) % 6] if n > 1 else 40 for i in range(n)]
    off = [0]
    for x in adds:
        off.append(off[-1] + x)
    c, m = make(layers=1, pages=2 * n + 3, heads=1, slots=n, width=3)
    seqs = list(range(n))[::-1]
    extend(c, m, seqs, off)
    append(c, m, seqs, off, False, (0,))
    append(c, m, seqs, off, True, (0,))
    assert c.status() == 0
