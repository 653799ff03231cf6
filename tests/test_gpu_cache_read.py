"""Rows read out of a cache of 16-bit pages: the bits that were appended, wherever they lie."""
import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def bits(x):
    return x.contiguous().view(torch.int16)


def rows(n, heads, dim, act, seed):
    """Any bits, infinities and NaN among them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-2 ** 15, 2 ** 15, (n, heads, dim), generator=g, device="cuda", dtype=torch.int16).view(act)


def filled(act, heads, dim, page, lens, layer=1):
    """A cache whose slot i holds lens[i] tokens, appended in two pieces, and their K and V."""
    n = len(lens)
    pages = sum(-(-x // page) for x in lens) + 9
    shape = (2, pages, page, heads, dim)
    c = tfx.Cache(torch.empty(shape, dtype=act, device="cuda"), torch.empty(shape, dtype=act, device="cuda"), n + 2, max(lens) // page + 2)
    tfx.cache_reserve(c, n + 2, heads)
    held = [[], []]
    first = [x // 3 for x in lens]
    for part, adds in enumerate((first, [a - b for a, b in zip(lens, first)])):
        at = [0]
        for x in adds:
            at.append(at[-1] + x)
        kv = [rows(at[-1], heads, dim, act, 10 * part + i) for i in range(2)]
        tfx.cache_extend(c, dev(range(n)), dev(at))
        tfx.cache_append(c, layer, *kv)
        for h, x in zip(held, kv):
            h.append([x[a:b] for a, b in zip(at, at[1:])])
    return c, [[torch.cat([h[0][i], h[1][i]]) for i in range(n)] for h in held]


@pytest.mark.parametrize("act", [F16, BF16])
@pytest.mark.parametrize("heads,dim,page", [(1, 128, 16), (3, 128, 32), (5, 256, 64), (8, 128, 128), (2, 256, 16)])
def test_rows_of_16_bit_pages(act, heads, dim, page):
    """Whole sequences, parts that begin and end inside pages, a sequence twice, none; into slices of a wider buffer, of which
    the rest stays; out of forks and after a compaction."""
    lens = [300, 1, 129, 64, 0, 17]
    c, held = filled(act, heads, dim, page, lens)
    tfx.cache_fork(c, dev([2]), dev([6]))
    tfx.cache_free(c, dev([0]))
    tfx.cache_compact(c)
    for h in held:
        h.append(h[2])
    parts = [(2, 0, 129), (6, 100, 29), (5, 3, 14), (4, 0, 0), (1, 0, 1), (2, 15, 2), (3, 0, 64), (3, 63, 1)]
    at = [2]
    for _, _, n in parts:
        at.append(at[-1] + n)
    total = at[-1] + 3
    buf = torch.full((2, total, heads * dim + 16), 5.0, dtype=act, device="cuda")
    out = tuple(b[:, 8:8 + heads * dim].unflatten(1, (heads, dim)) for b in buf)
    got = tfx.cache_read(c, 1, dev(p[0] for p in parts), dev(p[1] for p in parts), dev(at), at[-1], out=out)
    assert c.status() == 0
    want = torch.full((2, total, heads, dim), 5.0, dtype=act, device="cuda")
    for h, w in zip(held, want):
        for (s, a, n), b in zip(parts, at):
            w[b:b + n] = h[s][a:a + n]
    for g, w in zip(got, want):
        assert torch.equal(bits(g), bits(w))
    assert bool((buf[:, :, :8] == 5).all()) and bool((buf[:, :, 8 + heads * dim:] == 5).all())
    made = tfx.cache_read(c, 1, dev(p[0] for p in parts), dev(p[1] for p in parts), dev(at), total)
    for g, w in zip(made, want):
        assert torch.equal(bits(g[2:at[-1]]), bits(w[2:at[-1]])) and not bits(g[:2]).any() and not bits(g[at[-1]:]).any()


@pytest.mark.parametrize("act", [F16, BF16])
def test_many_rows_of_16_bit_pages(act):
    """As many rows as give a task 2, 4 and 8 tokens."""
    lens = [5000, 12345, 16, 33]
    c, held = filled(act, 4, 256, 64, lens)
    for n in (40, 700, 2000, 5000, 12345):
        for start in (0, 7, 12345 - n):
            if start + n <= 12345:
                k, v = tfx.cache_read(c, 1, dev([1]), dev([start]), dev([0, n]), n)
                assert torch.equal(bits(k), bits(held[0][1][start:start + n])) and torch.equal(bits(v), bits(held[1][1][start:start + n]))
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    k, v = tfx.cache_read(c, 1, dev(range(4)), dev([0] * 4), dev(at), at[-1])
    assert torch.equal(bits(k), bits(torch.cat(held[0]))) and torch.equal(bits(v), bits(torch.cat(held[1]))) and c.status() == 0
