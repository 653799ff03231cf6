"""A cache of 8-bit codes: appends, reads, page operations and attention against tests/q8_reference.py."""
import numpy as np
import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx
from q8_reference import BLOCK, TOP, Coded, assert_near, attend

pytestmark = pytest.mark.gpu
F16, BF16, I8, E4M3 = torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn
STORES = [I8, E4M3]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def keys(shape, dtype, seed):
    """Sizes that differ from channel to channel and from token to token, as a model's do."""
    x = normal(shape, torch.float32, seed)
    x[..., 3::37] *= 12
    return (x * torch.exp2(torch.randint(-6, 7, (shape[0], 1, 1), generator=torch.Generator().manual_seed(seed)).float().cuda())).to(dtype)


def make(store, act=F16, layers=2, pages=12, page=32, heads=2, dim=256, slots=4, width=8, batch=4, hq=8, fill=0x7F):
    """Pages and scales that hold NaN (of E4M3) and junk before anything is written."""
    shape = (layers, pages, page, heads, dim)
    k, v = (torch.full(shape, fill, dtype=torch.uint8, device="cuda").view(store) for _ in range(2))
    ks, vs = (torch.full((layers, pages, page // BLOCK, heads), float("nan"), device="cuda") for _ in range(2))
    c = tfx.Cache(k, v, slots, width, k_scale=ks, v_scale=vs, act=act)
    tfx.cache_reserve(c, max_batch=batch, heads=hq)
    return c


class Model:
    """What each sequence holds, beside the cache."""

    def __init__(self, c, store):
        self.c, self.store = c, store
        self.seqs = {}

    def put(self, layer, adds, seed, scale=1.0):
        """One extend and append: adds is {slot: tokens}."""
        c = self.c
        slots, lens = list(adds), list(adds.values())
        at = np.concatenate([[0], np.cumsum(lens)]).tolist()
        seqs, off = dev(*slots), dev(*at)
        k, v = (keys((at[-1], c.heads_kv, c.dim), c.dtype, seed + i) * scale for i in range(2))
        tfx.cache_extend(c, seqs, off)
        tfx.cache_append(c, layer, k, v)
        for i, s in enumerate(slots):
            pair = self.seqs.setdefault(s, [Coded(self.store, c.heads_kv, c.dim) for _ in range(2)])
            for m, x in zip(pair, (k, v)):
                m.append(x[at[i]:at[i + 1]].double().cpu().numpy())
        return k, v

    def check(self, layer):
        """Codes and scales of every token that is held, and zero status."""
        c = self.c
        lens, tables = c.lens.tolist(), c.tables.tolist()
        for s, pair in self.seqs.items():
            n = len(pair[0].codes)
            assert lens[s] == n
            used = torch.tensor(tables[s][:-(-n // c.s.page_size)], dtype=torch.long, device="cuda")
            for m, pool, scales in zip(pair, (c.k, c.v), (c.k_scale, c.v_scale)):
                got = pool[layer].view(torch.uint8)[used].view(pool.dtype).float().reshape(-1, c.heads_kv, c.dim)[:n]
                sc = scales[layer][used].reshape(-1, c.heads_kv)[:-(-n // BLOCK)].double().cpu().numpy()
                assert np.array_equal(sc, m.scales, equal_nan=True)
                bad = np.repeat(np.isnan(m.scales), BLOCK, 0)[:n]
                got = got.double().cpu().numpy()
                assert np.array_equal(got[~bad], m.codes[~bad])
        assert c.status() == 0


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("act,heads,dim,page", [(F16, 2, 256, 32), (BF16, 1, 128, 16), (BF16, 5, 256, 64), (F16, 9, 128, 128)])
def test_appends_bytes(store, act, heads, dim, page):
    """Prompts, single tokens whose size grows and shrinks, blocks that end inside a page and at its end."""
    c = make(store, act, pages=40, page=page, heads=heads, dim=dim, width=9, hq=heads)
    m = Model(c, store)
    m.put(1, {2: 37, 0: 1, 3: 16}, 1)
    m.check(1)
    for step, scale in enumerate([1.0, 4.0, 0.25, 37.0, 1.0, 300.0]):
        m.put(1, {0: 1, 2: 1, 3: 1}, 10 + 2 * step, scale)
    m.check(1)
    m.put(1, {0: 0, 3: 23, 1: 5}, 50)
    m.put(1, {1: 11, 2: 2}, 60, 0.01)
    m.check(1)
    m.put(1, {1: 1}, 70)
    m.check(1)
    assert bool((c.k[0].view(torch.uint8) == 0x7F).all()) and bool(c.k_scale[0].isnan().all())  # the other layer


@pytest.mark.parametrize("store", STORES)
def test_append_of_extreme_values(store):
    """Zeros, the type's smallest and largest values, the codes' border, ties."""
    c = make(store, BF16, heads=1, dim=128)
    top = TOP[store]
    x = torch.zeros((7 * 16, 1, 128), dtype=BF16, device="cuda")
    x[16:32] = 2.0 ** -133
    x[32:48] = torch.finfo(BF16).max
    x[48:64] = top * 2.0 ** -3
    x[64, 0, 0], x[65] = top * 2, (torch.arange(128, device="cuda") * 0.5).to(BF16)[None]
    x[80, 0, :], x[95, 0, 5] = 2.0 ** -9, top
    x[96, 0, 0] = top * 1.01 if store == I8 else top * 1.0078125
    off = dev(0, x.shape[0])
    tfx.cache_extend(c, dev(1), off)
    tfx.cache_append(c, 0, x, -x)
    m = Model(c, store)
    m.seqs[1] = [Coded(store, 1, 128), Coded(store, 1, 128)]
    m.seqs[1][0].append(x.double().cpu().numpy())
    m.seqs[1][1].append(-x.double().cpu().numpy())
    m.check(0)


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite(store, what):
    """Their block is NaN (and stays it until its page is taken anew), the others are as they were."""
    c = make(store)
    m = Model(c, store)
    m.put(0, {0: 20, 1: 20}, 3)
    k, v = normal((1, 2, 256), F16, 1), normal((1, 2, 256), F16, 2)
    k[0, 1, 77] = what
    tfx.cache_extend(c, dev(0), dev(0, 1))
    tfx.cache_append(c, 0, k, v)
    for x, pair in zip((k, v), m.seqs[0]):
        pair.append(x.double().cpu().numpy())
    m.put(0, {0: 3, 1: 5}, 4)
    m.check(0)
    got, _ = tfx.cache_read(c, 0, dev(0), dev(0), dev(0, 24), 24)
    assert bool(got[16:, 1].isnan().all()) and not bool(got[:16].isnan().any()) and not bool(got[:, 0].isnan().any())
    q = normal((2, 8, 256), F16, 9)
    out = tfx.attn_decode(c, 0, q, dev(0, 1))
    assert bool(out[0, 4:].isnan().all()) and bool(out[0, :4].isfinite().all()) and bool(out[1].isfinite().all())
    tfx.cache_free(c, dev(0))
    m.seqs.pop(0)
    m.put(0, {0: 40}, 5)
    m.check(0)


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("act", [F16, BF16])
@pytest.mark.parametrize("dim,heads,page", [(256, 3, 16), (128, 4, 64)])
def test_read(store, act, dim, heads, page):
    """Whole sequences, parts, one twice, none; rows outside the lists and past `rows` stay."""
    c = make(store, act, pages=30, page=page, heads=heads, dim=dim, hq=heads)
    m = Model(c, store)
    m.put(1, {0: 70, 2: 1, 3: 45}, 1)
    m.put(1, {0: 3, 2: 30}, 5)
    parts = [(0, 0, 73), (3, 17, 5), (3, 17, 5), (2, 30, 1), (1, 0, 0), (0, 15, 34)]
    at = np.concatenate([[2], 2 + np.cumsum([n for _, _, n in parts])]).tolist()
    rows = at[-1] + 3
    buf = torch.full((2, rows, heads * dim + 8), 5.0, dtype=act, device="cuda")
    out = tuple(b[:, :heads * dim].unflatten(1, (heads, dim)) for b in buf)
    k, v = tfx.cache_read(c, 1, dev(*[p[0] for p in parts]), dev(*[p[1] for p in parts]), dev(*at), at[-1] - 1, out=out)
    assert k.data_ptr() == out[0].data_ptr()
    for x, which in ((k, 0), (v, 1)):
        for (s, a, n), b in zip(parts, at):
            n = min(n, at[-1] - 1 - b)
            if n > 0:
                want = torch.tensor(m.seqs[s][which].values()[a:a + n]).to(act)
                assert torch.equal(x[b:b + n].cpu(), want)
        assert bool((x[:2] == 5).all()) and bool((x[at[-1] - 1:] == 5).all())
    assert bool((buf[:, :, heads * dim:] == 5).all()) and c.status() == 0


@pytest.mark.parametrize("store", [F16, I8])
def test_read_of_what_is_not_held(store):
    """Zeros and a status bit: past the end, before the start, a slot out of range, an empty slot."""
    if store == F16:
        k = normal((1, 6, 16, 2, 128), F16, 1)
        c = tfx.Cache(k, k.clone(), 3, 4)
        tfx.cache_reserve(c, 1, 2)
        x = normal((20, 2, 128), F16, 3)
        tfx.cache_extend(c, dev(1), dev(0, 20))
        tfx.cache_append(c, 0, x, -x)
        want = x
    else:
        c = make(store, layers=1, pages=6, page=16, dim=128, slots=3, width=4)
        m = Model(c, store)
        m.put(0, {1: 20}, 3)
        want = torch.tensor(m.seqs[1][0].values()).half().cuda()
    seqs, starts, at = dev(1, 1, -1, 3, 0, 1, 1), dev(18, -1, 0, 0, 0, 2 ** 31 - 1, 0), dev(0, 4, 6, 8, 10, 11, 12, 14)
    k, _ = tfx.cache_read(c, 0, seqs, starts, at, 20)
    assert c.status() == tfx.CACHE_BAD
    zero = torch.ones(20, dtype=torch.bool)
    zero[[0, 1, 5, 12, 13]] = False
    assert bool((k[zero.cuda()] == 0).all())
    assert torch.equal(k[[0, 1, 5, 12, 13]], want[[18, 19, 0, 0, 1]])


@pytest.mark.parametrize("store", STORES)
def test_page_operations_take_scales_along(store):
    c = make(store, pages=20, slots=6, width=5, page=32)
    m = Model(c, store)
    for layer in (0, 1):
        if layer:
            tfx.cache_append(c, 1, *new, dev(0, 1), dev(0, 75, 145))
        else:
            new = m.put(0, {0: 75, 1: 70}, 1)
    tfx.cache_fork(c, dev(0, 1, 0), dev(2, 3, 4))
    for s, d in ((0, 2), (1, 3), (0, 4)):
        m.seqs[d] = [Coded(store, 2, 256) for _ in range(2)]
        for a, b in zip(m.seqs[s], m.seqs[d]):
            b.codes, b.scales = a.codes.copy(), a.scales.copy()
    m.check(0)
    m.check(1)
    seqs = dict(m.seqs)
    m.put(0, {2: 1, 3: 7, 4: 2, 0: 1}, 7, 50.0)  # each grows its own copy of the last page
    m.check(0)
    tfx.cache_free(c, dev(1, 4))
    for s in (1, 4):
        m.seqs.pop(s)
    tfx.cache_compact(c)
    assert int(c.book[1]) > 0
    m.check(0)
    used = sorted({p for row in c.tables.tolist() for p in row if p >= 0})
    free = [p for p in range(20) if p not in used][:2]
    tfx.cache_copy(c, dev(used[0], used[1]), dev(*free))
    for x in (c.k_scale, c.v_scale):
        a, b = x[:, used[:2]], x[:, free]
        assert bool(((a == b) | (a.isnan() & b.isnan())).all())
    assert torch.equal(c.k.view(torch.uint8)[:, used[:2]], c.k.view(torch.uint8)[:, free])


def check_decode(c, m, layer, q, seqs, shared, got, scale):
    group = q.shape[1] // c.heads_kv
    cut = shared // BLOCK * BLOCK
    first = next((s for s in seqs if s in m.seqs and len(m.seqs[s][0].codes) >= shared), None)
    for i, s in enumerate(seqs):
        if s not in m.seqs or not len(m.seqs[s][0].codes):
            assert bool((got[i] == 0).all())
            continue
        k, v = (torch.tensor(x.values()).cuda() for x in m.seqs[s])
        n = min(cut, k.shape[0])
        if n:
            fk, fv = (torch.tensor(x.values()[:n]).cuda() for x in m.seqs[first])
            k, v = torch.cat([fk, k[n:]]), torch.cat([fv, v[n:]])
        most = TOP[m.store] * max(x[1].scales.max() for x in m.seqs.values() if len(x[1].scales))
        for h in range(q.shape[1]):
            o, A, qk = attend(q[i, h:h + 1], k[:, h // group], v[:, h // group], scale)
            assert_near(got[i:i + 1, h], o, A, qk, k.shape[0], c.dim, most)


DECODES = [
    # heads, kv heads, dim, page, lengths
    (8, 2, 256, 32, [1, 17, 0, 300]),
    (24, 4, 256, 16, [1000]),
    (7, 1, 128, 64, [33, 1, 64, 65, 16, 15, 31, 32]),
    (16, 1, 128, 16, [129, 511]),
    (20, 2, 256, 128, [2, 140]),
    (18, 1, 256, 16, [47, 16]),
    (6, 6, 128, 32, [700, 5]),
    (100, 1, 128, 64, [100, 3]),
]


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("act", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,dim,page,lens", DECODES)
def test_decode(store, act, hq, hkv, dim, page, lens):
    pages = sum(-(-n // page) for n in lens) + 3
    c = make(store, act, layers=1, pages=pages, page=page, heads=hkv, dim=dim, slots=len(lens) + 1,
             width=-(-max(lens) // page) + 1, batch=len(lens) + 2, hq=hq)
    m = Model(c, store)
    m.put(0, {i: n for i, n in enumerate(lens)}, 2)
    m.put(0, {i: 1 for i, n in enumerate(lens) if n}, 4, 2.0)
    order = list(range(len(lens)))[::-1] + [-1, len(lens)]  # a slot out of range, an empty one
    q = normal((len(order), hq, dim), act, 7, 0.3)
    got = tfx.attn_decode(c, 0, q, dev(*order))
    check_decode(c, m, 0, q, order, 0, got, dim ** -0.5)
    assert tfx.attn_error() == 0


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("hq,hkv,dim,page,shared,own", [
    (8, 2, 256, 32, 100, [1, 40, 17]), (24, 4, 256, 16, 15, [3, 1]), (12, 2, 128, 64, 515, [1] * 9), (5, 1, 128, 16, 48, [1, 70, 2]),
    (32, 1, 256, 128, 384, [5, 1, 1]), (2, 2, 128, 32, 33, [1] * 40)])
def test_decode_behind_a_shared_prefix(store, hq, hkv, dim, page, shared, own):
    n = len(own)
    width = -(-(shared + max(own)) // page) + 1
    c = make(store, BF16, layers=1, pages=width * (n + 1), page=page, heads=hkv, dim=dim, slots=n + 1, width=width, batch=n, hq=hq)
    m = Model(c, store)
    m.put(0, {n: shared}, 2)
    tfx.cache_fork(c, dev(*[n] * n), dev(*range(n)))
    for i in range(n):
        m.seqs[i] = [Coded(store, hkv, dim) for _ in range(2)]
        for a, b in zip(m.seqs[n], m.seqs[i]):
            b.codes, b.scales = a.codes.copy(), a.scales.copy()
    m.put(0, {i: x for i, x in enumerate(own)}, 4, 3.0)
    q = normal((n, hq, dim), BF16, 7, 0.3)
    got = tfx.attn_decode(c, 0, q, dev(*range(n)), shared=shared)
    check_decode(c, m, 0, q, list(range(n)), shared, got, dim ** -0.5)


@pytest.mark.parametrize("store", STORES)
def test_decode_of_values_with_very_different_scales(store):
    """The scales of V reach from 2^-126 (a block of zeros) to the largest; the heaviest keys are not the largest values."""
    c = make(store, BF16, layers=1, page=16, heads=1, dim=128, pages=12, width=11)
    m = Model(c, store)
    n = 160
    k, v = normal((n, 1, 128), BF16, 1), normal((n, 1, 128), BF16, 2)
    v[:16] = 0
    for b, e in enumerate([-30, 0, 20, -12, 5, -3, 40, 0, -20], 1):
        v[16 * b:16 * b + 16] *= 2.0 ** e
    q = normal((1, 4, 128), BF16, 3)
    k[16 * 7:16 * 8] = q[0, 0].float().mul(0.0).to(BF16) - 9 * q[0, :1]  # the block of 2^40 has no weight for head 0
    k[3] = 2 * q[0, 1]  # head 1 looks at the zeros
    tfx.cache_extend(c, dev(0), dev(0, n))
    tfx.cache_append(c, 0, k, v)
    m.seqs[0] = [Coded(store, 1, 128) for _ in range(2)]
    for x, y in zip(m.seqs[0], (k, v)):
        x.append(y.double().cpu().numpy())
    got = tfx.attn_decode(c, 0, q, dev(0), scale=1.0)
    kk, vv = (torch.tensor(x.values()).cuda()[:, 0] for x in m.seqs[0])
    for h in range(4):
        o, A, qk = attend(q[0, h:h + 1], kk, vv, 1.0)
        # of each row, what its own weights leave: the largest scale that counts for FP16's steps is under 2^-p of the row's A
        p = torch.softmax(q[0, h:h + 1].double() @ kk.T, 1)[0]
        most = TOP[store] * float((p.view(-1, 16).amax(1).cpu() * torch.tensor(m.seqs[0][1].scales[:, 0])).max())
        assert_near(got[:, h], o, A, qk, n, 128, most)


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("act,hq,hkv,dim,page,shared,n", [
    (BF16, 24, 4, 256, 64, 1000, 30), (F16, 8, 1, 128, 16, 703, 17), (F16, 128, 1, 256, 32, 320, 2), (BF16, 6, 2, 128, 128, 5000, 64),
    (F16, 16, 16, 128, 16, 300, 40), (BF16, 20, 1, 256, 16, 256, 7), (F16, 12, 2, 256, 64, 575, 70)])
def test_decode_of_many_rows_behind_a_prefix(store, act, hq, hkv, dim, page, shared, n):
    """Rows that fill several tiles and part of one, shares of the prefix, sequences that end inside it and one that is empty."""
    width = shared // page + 2
    c = make(store, act, layers=1, pages=width * 2 + n * 2 + 4, page=page, heads=hkv, dim=dim, slots=n + 4, width=width, batch=n + 3, hq=hq)
    m = Model(c, store)
    m.put(0, {n: shared}, 2)
    tfx.cache_fork(c, dev(*[n] * n), dev(*range(n)))
    for i in range(n):
        m.seqs[i] = [Coded(store, hkv, dim) for _ in range(2)]
        for a, b in zip(m.seqs[n], m.seqs[i]):
            b.codes, b.scales = a.codes.copy(), a.scales.copy()
    m.put(0, {i: 1 + i % 3 for i in range(n)}, 4, 3.0)
    # shorter ones: the prefix's first tokens
    for slot, held in ((n + 1, 100), (n + 2, 17)):
        m.seqs[slot] = [Coded(store, hkv, dim) for _ in range(2)]
        for a, b in zip(m.seqs[n], m.seqs[slot]):
            b.codes, b.scales = a.codes[:held].copy(), a.scales[:-(-held // BLOCK)].copy()
        c.lens[slot] = held
        c.tables[slot] = c.tables[n]
    order = list(range(n)) + [n + 1, n + 2, n + 3]
    q = normal((n + 3, hq, dim), act, 7, 0.3)
    got = tfx.attn_decode(c, 0, q, dev(*order), shared=shared)
    assert tfx.attn_error() == 0
    check_decode(c, m, 0, q, order, shared, got, dim ** -0.5)


@pytest.mark.parametrize("store", STORES)
def test_prefix_of_values_with_very_different_scales(store):
    """As test_decode_of_values_with_very_different_scales, in the prefix of a batch; scales of 2^100 that have next to no weight."""
    n, batch = 512, 16
    c = make(store, BF16, layers=1, page=64, heads=1, dim=128, pages=30, width=12, slots=batch + 1, batch=batch, hq=4)
    k, v = normal((n, 1, 128), BF16, 1), normal((n, 1, 128), BF16, 2)
    q = normal((batch, 4, 128), BF16, 3)
    v[:16] = 0
    for b in range(1, n // 16):
        v[16 * b:16 * b + 16] *= 2.0 ** ((b * 37) % 61 - 30)
    v[160:176] *= 2.0 ** 100
    k[160:176] = q[:, 0].float().mean(0).to(BF16) * -40
    k[3] = 2 * q[0, 1]
    tfx.cache_extend(c, dev(batch), dev(0, n))
    tfx.cache_append(c, 0, k, v)
    tfx.cache_fork(c, dev(*[batch] * batch), dev(*range(batch)))
    pair = [Coded(store, 1, 128) for _ in range(2)]
    for x, y in zip(pair, (k, v)):
        x.append(y.double().cpu().numpy())
    got = tfx.attn_decode(c, 0, q, dev(*range(batch)), shared=n, scale=1.0)
    kk, vv = (torch.tensor(x.values()).cuda()[:, 0] for x in pair)
    scales = torch.tensor(pair[1].scales[:, 0])
    for i in range(batch):
        for h in range(4):
            o, A, qk = attend(q[i, h:h + 1], kk, vv, 1.0)
            p = torch.softmax(q[i, h:h + 1].double() @ kk.T, 1)[0]
            most = TOP[store] * float((p.view(-1, 16).amax(1).cpu() * scales).max())
            assert_near(got[i:i + 1, h], o, A, qk, n, 128, most)


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("dim,page", [(128, 32), (256, 16)])
@pytest.mark.parametrize("rise,grow", [(7.9, 0), (8.2, 0), (0.6, 0), (-2.0, 8), (4.0, 4), (0.0, 7), (3.0, -11)])
def test_scores_and_values_that_rise_from_block_to_block(store, dim, page, rise, grow):
    """By less and by more than what moves the references: log2 of a weight by `rise`, of a value by `grow`."""
    n = 16 * 12
    c = make(store, F16, layers=1, page=page, heads=1, dim=dim, pages=n // page + 1, width=n // page)
    m = Model(c, store)
    k, v = normal((n, 1, dim), F16, 1, 0.05), normal((n, 1, dim), F16, 2, 2.0 ** -8 if grow > 0 else 1.0)
    block = torch.arange(n, device="cuda") // 16
    k[:, 0, 0] = (block - 6) * rise * float(np.log(2))
    v = (v.float() * torch.exp2(block.float().clamp(max=2) * grow)[:, None, None]).to(F16)  # the factor alone passes FP16's range
    q = normal((1, 3, dim), F16, 3, 0.1)
    q[0, :, 0] = torch.tensor([1.0, -1.0, 0.5])
    tfx.cache_extend(c, dev(0), dev(0, n))
    tfx.cache_append(c, 0, k, v)
    m.seqs[0] = [Coded(store, 1, dim) for _ in range(2)]
    for x, y in zip(m.seqs[0], (k, v)):
        x.append(y.double().cpu().numpy())
    got = tfx.attn_decode(c, 0, q, dev(0), scale=1.0)
    kk, vv = (torch.tensor(x.values()).cuda()[:, 0] for x in m.seqs[0])
    for h in range(3):
        o, A, qk = attend(q[0, h:h + 1], kk, vv, 1.0)
        # what counts for FP16's steps: as above, the largest product of a weight and a scale
        p = torch.softmax(q[0, h:h + 1].double() @ kk.T, 1)[0]
        most = TOP[store] * float((p.view(-1, 16).amax(1).cpu() * torch.tensor(m.seqs[0][1].scales[:, 0])).max())
        assert_near(got[:, h], o, A, qk, n, dim, most)
    assert tfx.attn_error() == 0
