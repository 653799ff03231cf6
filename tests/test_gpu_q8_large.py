"""8-bit caches where sizes decide: prefixes that the tensor cores read once, pools and rows past 2^32
elements, streams, captured graphs, bounded waits, calls that share a cache."""
import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx
from q8_reference import BLOCK, TOP, assert_near, attend

pytestmark = pytest.mark.gpu
F16, BF16, I8, E4M3 = torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def make(store, act, pages, page, heads, dim, slots, width, batch, hq, layers=1):
    """Pages and scales that hold NaN (of E4M3) and junk before anything is written."""
    k, v = (torch.full((layers, pages, page, heads, dim), 0x7F, dtype=torch.uint8, device="cuda").view(store) for _ in range(2))
    ks, vs = (torch.full((layers, pages, page // BLOCK, heads), float("nan"), device="cuda") for _ in range(2))
    c = tfx.Cache(k, v, slots, width, k_scale=ks, v_scale=vs, act=act)
    tfx.cache_reserve(c, batch, hq)
    return c


def put(c, adds, seed, vscale=None):
    """One extend and append: adds is [(slot, tokens)]."""
    at = [0]
    for _, n in adds:
        at.append(at[-1] + n)
    k, v = (normal((at[-1], c.heads_kv, c.dim), c.dtype, seed + i) for i in range(2))
    if vscale is not None:
        v = (v.float() * vscale[:, None, None]).to(c.dtype)
    tfx.cache_extend(c, dev(s for s, _ in adds), dev(at))
    tfx.cache_append(c, 0, k, v)


def values(c, slot, n, start=0):
    """The values that codes and scales stand for, by torch."""
    page = c.s.page_size
    used = c.tables[slot, start // page:-(-n // page)].long()
    out = []
    for pool, scales in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x = pool[0].view(torch.uint8)[used].view(pool.dtype).double().view(-1, page // BLOCK, BLOCK, c.heads_kv, c.dim)
        x = x * scales[0][used].double()[:, :, None, :, None]
        out.append(x.reshape(-1, c.heads_kv, c.dim)[start % page:n - start // page * page])
    return out


def behind(c, n, shared, batch, own, short=()):
    """Slot n holds a prefix of `shared` tokens, slots 0 .. n-1 fork it and take own(i) tokens more;
    slots from n+1 on hold the prefix's first tokens."""
    put(c, [(n, shared)], 1)
    tfx.cache_fork(c, dev([n] * n), dev(range(n)))
    put(c, [(i, own(i)) for i in range(n)], 3)
    for i, held in enumerate(short):
        c.lens[n + 1 + i] = held
        c.tables[n + 1 + i] = c.tables[n]
    assert c.status() == 0


def check(c, q, seqs, got, shared, prefix_of, scale, most=None):
    group, cut = q.shape[1] // c.heads_kv, shared // BLOCK * BLOCK
    lens = c.lens.tolist()
    fk, fv = values(c, prefix_of, cut) if cut else (None, None)
    for i, s in enumerate(seqs):
        n = lens[s]
        if n == 0:
            assert bool((got[i] == 0).all())
            continue
        if cut and n > cut:
            k, v = values(c, s, n, cut)
            k, v = torch.cat([fk, k]), torch.cat([fv, v])
        else:
            k, v = (fk[:n], fv[:n]) if cut else values(c, s, n)
        top = most or TOP[c.k.dtype] * float(c.v_scale[c.v_scale.isfinite()].max())
        for h in range(c.heads_kv):
            rows = slice(h * group, (h + 1) * group)
            o, A, qk = attend(q[i, rows], k[:, h], v[:, h], scale)
            assert_near(got[i, rows], o, A, qk, k.shape[0], c.dim, top)


PREFIXES = [  # batch * shared tokens take more than 64 MiB
    (BF16, E4M3, 24, 4, 256, 64, 1205, 30), (F16, I8, 8, 1, 128, 16, 2711, 100), (F16, E4M3, 128, 1, 256, 32, 13201, 10),
    (BF16, I8, 16, 16, 128, 16, 430, 40), (BF16, E4M3, 20, 1, 256, 128, 2100, 64), (F16, I8, 6, 2, 128, 128, 5000, 64),
    (BF16, I8, 24, 4, 256, 16, 11007, 3), (F16, I8, 4, 1, 256, 64, 1000, 140)]


@pytest.mark.parametrize("act,store,hq,hkv,dim,page,shared,n", PREFIXES)
def test_a_prefix_read_once(act, store, hq, hkv, dim, page, shared, n):
    """Tiles of 128 rows, whole and partly filled, shares of the prefix, sequences that end inside it, an empty one."""
    width = shared // page + 4
    c = make(store, act, width + 4 * n, page, hkv, dim, n + 4, width, n + 3, hq)
    behind(c, n, shared, n, lambda i: 1 + i % 19, (100, 17))
    order = list(range(n)) + [n + 1, n + 2, n + 3]
    q = normal((n + 3, hq, dim), act, 7, 0.3)
    got = tfx.attn_decode(c, 0, q, dev(order), shared=shared)
    assert tfx.attn_error() == 0
    check(c, q, order, got, shared, n, dim ** -0.5)
    alone = tfx.attn_decode(c, 0, q[:2], dev(order[:2]), shared=shared)  # two sequences read it as their own
    check(c, q[:2], order[:2], alone, shared, n, dim ** -0.5)


@pytest.mark.parametrize("store", [I8, E4M3])
def test_a_prefix_of_values_with_very_different_scales(store):
    """V's blocks from zeros to 2^100, the largest without weight: a block's factor leaves FP32's range, and its weights do not."""
    n, shared = 300, 912
    c = make(store, BF16, 64, 16, 1, 128, n + 1, 60, n, 4)  # forks share all its pages
    size = torch.exp2(((torch.arange(shared, device="cuda") // 16 * 37) % 61 - 30).float())
    size[:16], size[160:176] = 0, 2.0 ** 100
    g = normal((4, 128), BF16, 11)
    k = normal((shared, 1, 128), BF16, 1)
    k[160:176] = -40 * g[:1]
    k[3] = 2 * g[1]
    v = (normal((shared, 1, 128), BF16, 2).float() * size[:, None, None]).to(BF16)
    tfx.cache_extend(c, dev([n]), dev([0, shared]))
    tfx.cache_append(c, 0, k, v)
    tfx.cache_fork(c, dev([n] * n), dev(range(n)))
    assert c.status() == 0
    q = (g[None] + normal((n, 4, 128), BF16, 5, 0.05)).to(BF16)
    got = tfx.attn_decode(c, 0, q, dev(range(n)), shared=shared, scale=1.0)
    kk, vv = (x[:, 0] for x in values(c, n, shared))
    scales = c.v_scale[0][c.tables[n, :shared // 16].long()].double().reshape(-1)[:shared // 16]
    for i in range(0, n, 7):
        for h in range(4):
            o, A, qk = attend(q[i, h:h + 1], kk, vv, 1.0)
            p = torch.softmax(q[i, h:h + 1].double() @ kk.T, 1)[0]
            # the weights' steps are of the row's own largest weight: its probability times the scale of its block
            assert_near(got[i:i + 1, h], o, A, qk, shared, 128, TOP[store] * float((p.view(-1, 16).amax(1) * scales).max()),
                        float(vv.abs().max()))


def test_nan_in_a_prefix():
    """A NaN in one head's prefix reaches that head's rows of every sequence that sees it, and no others."""
    n, shared = 40, 900
    c = make(E4M3, F16, 200, 32, 4, 256, n + 2, 31, n + 1, 8)
    tfx.cache_extend(c, dev([n]), dev([0, shared]))
    k, v = normal((shared, 4, 256), F16, 1), normal((shared, 4, 256), F16, 2)
    v[500, 2, 7] = float("nan")
    tfx.cache_append(c, 0, k, v)
    tfx.cache_fork(c, dev([n] * n), dev(range(n)))
    assert c.status() == 0
    c.lens[n + 1] = 400  # ends before it
    c.tables[n + 1] = c.tables[n]
    got = tfx.attn_decode(c, 0, normal((n + 1, 8, 256), F16, 3), dev(list(range(n)) + [n + 1]), shared=shared)
    assert bool(got[:n, 4:6].isnan().all())
    assert bool(got[n].isfinite().all()) and bool(got[:, :4].isfinite().all()) and bool(got[:, 6:].isfinite().all())


@pytest.mark.parametrize("hq,hkv,dim,page,shared,n", [(24, 4, 256, 16, 0, 3), (8, 2, 128, 16, 0, 5), (24, 4, 256, 64, 1205, 30),
                                                     (6, 2, 128, 128, 5000, 64)])
def test_bounded_waits(hq, hkv, dim, page, shared, n):
    """A call that gives up says so, and the next one is right; the same bits every time."""
    width = (shared + 400) // page + 2
    c = make(I8, F16, width + n * (400 // page + 2), page, hkv, dim, n + 1, width, n, hq)
    if shared:
        behind(c, n, shared, n, lambda i: 1 + i % 19)
    else:
        put(c, [(i, 300 + i) for i in range(n)], 3)
    q, seqs = normal((n, hq, dim), F16, 7), dev(range(n))
    want = tfx.attn_decode(c, 0, q, seqs, shared=shared)
    for limit in (1, 300, 1500, 4000):
        tfx.set_spin_limit(limit)
        try:
            got = tfx.attn_decode(c, 0, q, seqs, shared=shared)
            assert tfx.attn_error() == 1 or torch.equal(got, want)
        finally:
            tfx.set_spin_limit(0)
        assert torch.equal(tfx.attn_decode(c, 0, q, seqs, shared=shared), want)
        assert tfx.attn_error() == 0


def test_a_step_in_a_graph_and_on_streams():
    """Rotation, extend, append, attention and read-back captured once and replayed: the same as call by call."""
    n, page, hq, hkv, dim = 6, 16, 12, 2, 256
    act, store = BF16, I8
    r = tfx.Rope(dim, 64)

    def caches():
        c = make(store, act, 80, page, hkv, dim, n, 12, n, hq)
        put(c, [(i, 10 + 13 * i) for i in range(n)], 3)
        return c

    a, b = caches(), caches()
    seqs, at = dev(range(n)), dev(range(n + 1))
    x = {name: normal((n, h, dim), act, 9 + h) for name, h in (("q", hq), ("k", hkv), ("v", hkv))}
    out = {}

    def step(c, where):
        tfx.cache_extend(c, seqs, at)
        positions = (c.lens[:n] - 1).contiguous()
        q, k = tfx.rope(r, x["q"], x["k"], positions, out=where["qk"])
        tfx.cache_append(c, 0, k, x["v"])
        tfx.attn_decode(c, 0, q, seqs, out=where["o"])
        tfx.cache_read(c, 0, seqs, positions, at, n, out=where["kv"])

    def places():
        e = lambda h: torch.zeros((n, h, dim), dtype=act, device="cuda")  # noqa: E731
        return {"qk": (e(hq), e(hkv)), "o": e(hq), "kv": (e(hkv), e(hkv))}

    wa, wb = places(), places()
    warm = caches()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm, places())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(b, wb)
    for i in range(5):
        x["q"].mul_(1.25)
        x["k"].mul_(1.5)  # the block's scale grows
        x["v"].neg_()
        step(a, wa)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip((*wa["qk"], wa["o"], *wa["kv"], a.book, a.k_scale.nan_to_num(), a.v_scale.nan_to_num()),
                        (*wb["qk"], wb["o"], *wb["kv"], b.book, b.k_scale.nan_to_num(), b.v_scale.nan_to_num())):
            assert torch.equal(u, v)
        assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8))
    assert a.status() == 0 and tfx.attn_error() == 0


def test_results_made_for_another_stream():
    """Results that a call makes are made, and cleared, in its stream's order."""
    c = make(I8, F16, 60, 16, 2, 128, 2, 40, 2, 4)
    put(c, [(0, 500), (1, 3)], 1)
    q, seqs = normal((2, 4, 128), F16, 5), dev([0, 1])
    r, at = tfx.Rope(128), dev([400, 2])
    want = (tfx.attn_decode(c, 0, q, seqs), *tfx.cache_read(c, 0, seqs, dev([0, 0]), dev([1, 301, 304]), 310), tfx.rope(r, q, None, at)[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.ones(1 << 28, device="cuda")
    for _ in range(20):
        big.mul_(1.0)  # the current stream is behind
    got = (tfx.attn_decode(c, 0, q, seqs, stream=side),
           *tfx.cache_read(c, 0, seqs, dev([0, 0]), dev([1, 301, 304]), 310, stream=side), tfx.rope(r, q, None, at, stream=side)[0])
    side.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    assert bool((got[1][0] == 0).all()) and bool((got[1][304:] == 0).all())


def test_a_pool_of_more_than_2_32_codes():
    """Pages whose codes begin past 2^32 bytes: append, read, attention by warps and by the prefix's kernel, copy."""
    page, hkv, dim = 128, 4, 256
    pages = (1 << 32) // (page * hkv * dim) + 700
    k, v = (torch.empty((1, pages, page, hkv, dim), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    n, shared = 40, 1000
    c = tfx.Cache(k, v, n + 1, 12, act=BF16)
    tfx.cache_reserve(c, n, 24)
    c.refs[:pages - 300] = 1  # in use by others
    behind(c, n, shared, n, lambda i: 1 + 5 * i)
    assert int(c.tables[n, 0]) >= pages - 300
    q = normal((n, 24, dim), BF16, 7, 0.3)
    got = tfx.attn_decode(c, 0, q, dev(range(n)), shared=shared)
    check(c, q, list(range(n)), got, shared, n, dim ** -0.5, TOP[E4M3] * float(c.v_scale[0, -300:].max()))
    got = tfx.attn_decode(c, 0, q[:2], dev(range(2)))
    check(c, q[:2], [0, 1], got, 0, n, dim ** -0.5, TOP[E4M3] * float(c.v_scale[0, -300:].max()))
    rk, rv = tfx.cache_read(c, 0, dev([39, n]), dev([0, 17]), dev([0, 1196, 1300]), 1300)
    wk, wv = values(c, 39, 1196)
    assert torch.equal(rk[:1196], wk.to(BF16)) and torch.equal(rv[:1196], wv.to(BF16))
    assert torch.equal(rk[1196:], values(c, n, 121, 17)[0].to(BF16))
    to = pages - 1
    tfx.cache_copy(c, c.tables[n, :1].clone(), dev([to]))
    assert torch.equal(c.k.view(torch.uint8)[0, to], c.k.view(torch.uint8)[0, int(c.tables[n, 0])])
    assert torch.equal(c.k_scale[0, to], c.k_scale[0, int(c.tables[n, 0])])


def test_rows_past_2_32_elements():
    """Rotation of the last rows of a tensor of more than 2^32 elements."""
    rows, pitch = 66000, 65536 + 64
    x = torch.empty((rows, pitch), dtype=F16, device="cuda")
    q = x[:, :256].unflatten(1, (2, 128))
    q[-3:] = normal((3, 2, 128), F16, 1)
    q[:3] = normal((3, 2, 128), F16, 2)
    at = torch.arange(rows, dtype=torch.int32, device="cuda")
    r = tfx.Rope(128)
    want = [tfx.rope(r, q[s].clone(), None, at[s])[0] for s in (slice(0, 3), slice(rows - 3, rows))]
    tfx.rope(r, q, None, at, out=(q, None))
    assert torch.equal(q[:3], want[0]) and torch.equal(q[-3:], want[1])


@pytest.mark.parametrize("n", [1, 31, 33, 200, 1500])
def test_lists_of_many_entries(n):
    """Appends and reads find their rows in lists with empty entries, in long runs too."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 4, (n,), generator=g)
    lens[n // 3:n // 3 + 70] = 0
    lens[-1] = 2
    c = make(I8, F16, n + 8, 16, 1, 128, n, 1, 1, 1)
    put(c, list(enumerate(lens.tolist())), 5)
    k, v = normal((int(lens.sum()), 1, 128), F16, 5), normal((int(lens.sum()), 1, 128), F16, 6)
    at = [0] + lens.cumsum(0).tolist()
    rk, rv = tfx.cache_read(c, 0, dev(range(n)), dev([0] * n), dev(at), at[-1])
    assert c.status() == 0
    # every row within half a step of its block's scale, which is at most amax / 63.5
    for got, x in ((rk, k), (rv, v)):
        step = torch.empty(at[-1], device="cuda")
        for a, b in zip(at, at[1:]):
            if b > a:
                step[a:b] = x[a:b].float().abs().max() / 63.5
        assert bool(((got.float() - x.float()).abs() <= step[:, None, None] * (0.5 + 2 ** -10)).all())


def test_a_batch_of_the_largest_size():
    c = make(E4M3, F16, 4100, 16, 1, 128, 4096, 2, 4096, 8)
    put(c, [(i, i % 16) for i in range(4096)], 3)
    q = normal((4096, 8, 128), F16, 5)
    got = tfx.attn_decode(c, 0, q, dev(range(4096)))
    some = list(range(0, 4096, 37)) + [4095]
    check(c, q[some], some, got[some], 0, 0, 128 ** -0.5)
