"""Attention through the public entry points against 64 bits (bound: attention_reference)."""
import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx
from attention_reference import assert_near, attend

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def offsets_of(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32)


def check_prompt(out, q, k, v, offsets, scale=None, heads=None):
    hq, dim = q.shape[1:]
    hkv = k.shape[1]
    scale = dim ** -0.5 if scale is None else scale
    at = offsets.tolist()
    for a, b in zip(at, at[1:]):
        if a == b:
            continue
        seen = torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").tril()
        for h in heads or range(hq):
            g = h // (hq // hkv)
            o, A, qk = attend(q[a:b, h], k[a:b, g], v[a:b, g], seen, scale)
            assert_near(out[a:b, h], o, A, qk, b - a, dim, q.dtype, float(v[a:b, g].abs().max()))


PROMPTS = [
    # heads, kv heads, dim, lens
    (24, 4, 256, [17]),
    (24, 4, 256, [1]),
    (6, 1, 256, [0, 1, 127, 128, 129, 0, 300, 21, 22, 43]),
    (48, 8, 128, [5, 255, 256, 257]),
    (16, 16, 128, [64, 1000]),
    (16, 1, 128, [9, 130]),
    (128, 1, 128, [3, 150]),
    (5, 1, 256, [77, 260]),
    (14, 2, 128, [513]),
    (96, 2, 256, [200]),
    (1, 1, 256, [384]),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,dim,lens", PROMPTS)
def test_prompt(dtype, hq, hkv, dim, lens):
    T = sum(lens)
    q, k, v = normal((T, hq, dim), dtype, 1, 1.5), normal((T, hkv, dim), dtype, 2), normal((T, hkv, dim), dtype, 3)
    off = offsets_of(lens)
    check_prompt(tfx.attn_prompt(q, k, v, off), q, k, v, off)


@pytest.mark.parametrize("dtype,dim", [(F16, 256), (BF16, 128)])
def test_long_prompt(dtype, dim):
    T = 5001
    q, k, v = normal((T, 12, dim), dtype, 1, 1.5), normal((T, 2, dim), dtype, 2), normal((T, 2, dim), dtype, 3)
    off = offsets_of([T])
    check_prompt(tfx.attn_prompt(q, k, v, off), q, k, v, off, heads=(0, 5, 11))


def test_many_sequences():
    """More sequences than one launch takes, most of them of a few tokens."""
    lens = [(i * 7) % 5 for i in range(1300)]
    T = sum(lens)
    q, k, v = normal((T, 4, 128), F16, 1), normal((T, 2, 128), F16, 2), normal((T, 2, 128), F16, 3)
    off = offsets_of(lens)
    check_prompt(tfx.attn_prompt(q, k, v, off), q, k, v, off, heads=(1, 2))


@pytest.mark.parametrize("dim", [128, 256])
def test_prompt_slices_of_one_buffer(dim):
    """q, k and v of one packed buffer with a pitch of its own, a scale, an output with a pitch, sequences that start late."""
    T, hq, hkv = 333, 12, 2
    x = normal((T, (hq + 2 * hkv) * dim + 8), BF16, 5)
    q = x[:, :hq * dim].unflatten(1, (hq, dim))
    k = x[:, hq * dim:(hq + hkv) * dim].unflatten(1, (hkv, dim))
    v = x[:, (hq + hkv) * dim:(hq + 2 * hkv) * dim].unflatten(1, (hkv, dim))
    buf = torch.full((T, hq * dim + 16), 7.0, dtype=BF16, device="cuda")
    out = buf[:, :hq * dim].unflatten(1, (hq, dim))
    off = offsets_of([100, 0, 150], 40)
    assert tfx.attn_prompt(q, k, v, off, scale=0.3, out=out) is out
    check_prompt(out, q, k, v, off, scale=0.3)
    assert bool((out[:40] == 7).all()) and bool((out[290:] == 7).all()) and bool((buf[:, hq * dim:] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 65504.0])
def test_prompt_other_rows_do_not_leak(bad):
    """Values of the rows around a sequence (other sequences, unused rows) change no bit of it."""
    lens, T = [50, 200, 61], 350
    q, k, v = normal((T, 6, 256), F16, 1), normal((T, 1, 256), F16, 2), normal((T, 1, 256), F16, 3)
    off = offsets_of(lens, 20)
    want = tfx.attn_prompt(q, k, v, off)[70:270].clone()
    for x in (q, k, v):
        x[:70] = bad
        x[270:] = bad
    assert torch.equal(tfx.attn_prompt(q, k, v, off)[70:270], want)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,dim", [(6, 1, 256), (8, 2, 128), (2, 2, 256)])
def test_prompt_later_values_do_not_reach_earlier_rows(hq, hkv, dim, dtype):
    """Infinite and NaN values of K and V are seen by their own and later rows only, and there as the formula has them."""
    T = 400
    q, k, v = normal((T, hq, dim), dtype, 1), normal((T, hkv, dim), dtype, 2), normal((T, hkv, dim), dtype, 3)
    off = offsets_of([10, 390])
    want = tfx.attn_prompt(q, k, v, off)
    v[140, 0, 5], v[141, 0, 5], v[150, 0, 7], v[155, 0, dim - 1] = float("inf"), -float("inf"), float("nan"), -float("inf")
    out = tfx.attn_prompt(q, k, v, off)
    assert torch.equal(out[:140], want[:140])
    g = hq // hkv
    assert bool((out[140, :g, 5] == float("inf")).all()) and out[141:, :g, 5].isnan().all()
    assert torch.equal(out[:150, :, 7], want[:150, :, 7]) and out[150:, :g, 7].isnan().all()
    assert bool((out[155:, :g, dim - 1] == -float("inf")).all())
    other = [c for c in range(dim) if c not in (5, 7, dim - 1)]
    assert torch.equal(out[:, :, other], want[:, :, other]) and torch.equal(out[:, g:], want[:, g:])
    v[:] = torch.nan_to_num(v, 0.0, 0.0, 0.0)
    want = tfx.attn_prompt(q, k, v, off)
    k[200, 0, 3] = float("nan")
    out = tfx.attn_prompt(q, k, v, off)
    assert torch.equal(out[:200], want[:200]) and out[200:, :g].isnan().all()


def test_prompt_sequence_bits_do_not_depend_on_the_call():
    lens = [300, 17, 129]
    T = sum(lens)
    q, k, v = normal((T, 24, 256), BF16, 1), normal((T, 4, 256), BF16, 2), normal((T, 4, 256), BF16, 3)
    out = tfx.attn_prompt(q, k, v, offsets_of(lens))
    assert torch.equal(out, tfx.attn_prompt(q, k, v, offsets_of(lens)))
    for i, n in enumerate(lens):
        a = sum(lens[:i])
        alone = tfx.attn_prompt(q[a:a + n], k[a:a + n], v[a:a + n], offsets_of([n]))
        assert torch.equal(out[a:a + n], alone)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompt_large_scores(dtype):
    """Scores of several hundred: the running maximum moves often and far."""
    T = 700
    q, k, v = normal((T, 6, 256), dtype, 1, 12.0), normal((T, 1, 256), dtype, 2, 4.0), normal((T, 1, 256), dtype, 3)
    ramp = torch.linspace(0.1, 3.0, T, device="cuda")[:, None, None].to(dtype)
    k = (k * ramp).contiguous()
    off = offsets_of([T])
    check_prompt(tfx.attn_prompt(q, k, v, off), q, k, v, off)


def test_prompt_equal_scores_give_the_mean():
    T = 400
    q = torch.zeros((T, 4, 128), dtype=F16, device="cuda")
    k, v = normal((T, 4, 128), F16, 2), normal((T, 4, 128), F16, 3)
    off = offsets_of([T])
    out = tfx.attn_prompt(q, k, v, off)
    check_prompt(out, q, k, v, off)
    assert torch.equal(out[0], v[0])


# ---- decode -----------------------------------------------------------------


def make_cache(lens, shared, page, hkv, dim, dtype, layers=1, extra=3, seed=0, poison=None):
    """Sequences of shared + lens[i] tokens that share their first full pages; scattered pages."""
    full = shared // page
    mine = [max(0, -(-(shared + n) // page) - full) if n >= 0 else 0 for n in lens]
    total = full + sum(mine) + extra
    g = torch.Generator()
    g.manual_seed(seed)
    numbers = torch.randperm(total, generator=g).tolist()
    width = full + max(mine) + 1
    k, v = normal((layers, total, page, hkv, dim), dtype, seed + 1), normal((layers, total, page, hkv, dim), dtype, seed + 2)
    c = tfx.Cache(k, v, len(lens), width)
    at, tables, refs = full, torch.full((len(lens), width), -1, dtype=torch.int32), torch.zeros(total, dtype=torch.int32)
    used = torch.zeros(total, page, dtype=torch.bool)
    for i, m in enumerate(mine):
        if lens[i] < 0:
            continue
        row = numbers[:full] + numbers[at:at + m]
        at += m
        tables[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
        for j, p in enumerate(row):
            refs[p] += 1
            used[p, :max(0, min(page, shared + lens[i] - j * page))] = True
        if shared % page and i:
            a, b = int(tables[0, full]), int(tables[i, full])
            for x in (k, v):
                x[:, b, :shared % page] = x[:, a, :shared % page]
    c.tables.copy_(tables)
    c.refs.copy_(refs)
    c.lens.copy_(torch.tensor([max(0, shared + n) if n >= 0 else 0 for n in lens], dtype=torch.int32))
    if poison is not None:
        free = (~used).to("cuda")
        for x in (k, v):
            x[:, free] = poison
    return c


def check_decode(out, c, layer, q, seqs, scale=None):
    hq, dim = q.shape[1:]
    hkv, page = c.s.heads_kv, c.s.page_size
    lens, tables = c.lens.tolist(), c.tables
    for i, s in enumerate(seqs.tolist()):
        n = lens[s]
        if n == 0:
            assert not out[i].any()
            continue
        at = tables[s, :-(-n // page)].long()
        k, v = (x[layer, at].reshape(-1, hkv, dim)[:n] for x in (c.k, c.v))
        seen = torch.ones(hq // hkv, n, dtype=torch.bool, device="cuda")
        for g in range(hkv):
            rows = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            o, A, qk = attend(q[i, rows], k[:, g], v[:, g], seen, dim ** -0.5 if scale is None else scale)
            assert_near(out[i, rows], o, A, qk, n, dim, q.dtype, float(v[:, g].abs().max()))


DECODES = [
    # heads, kv heads, dim, page, shared, lens (own tokens)
    (24, 4, 256, 16, 0, [1000]),
    (24, 4, 256, 16, 0, [1]),
    (24, 4, 256, 64, 0, [1, 0, 15, 16, 17, 200, 63, 64, 65]),
    (24, 4, 256, 16, 512, [1, 3, 100, 16]),
    (24, 4, 256, 64, 500, [1, 3, 100, 16, 700]),
    (24, 4, 256, 128, 1003, [0, 1, 300, 5]),
    (48, 8, 128, 32, 777, [9, 40, 1, 222, 31]),
    (48, 8, 128, 16, 1024, [5] * 23),
    (16, 16, 128, 16, 100, [33, 1, 64]),
    (16, 1, 128, 128, 3000, [33, 1, 640] * 7),
    (40, 1, 256, 64, 300, [90, 2]),
    (128, 1, 128, 64, 130, [90, 2, 31]),
    (28, 4, 128, 64, 4100, [77, 1, 2, 190] * 10),
    (6, 1, 256, 64, 2048, [(7 * i) % 90 + 1 for i in range(64)]),
    (24, 4, 256, 64, 9, [(7 * i) % 90 + 1 for i in range(70)]),
    (24, 4, 256, 128, 1100, [(5 * i) % 33 + 1 for i in range(45)]),
    (24, 4, 256, 16, 1003, [1] * 20),
    (12, 4, 256, 32, 300, [3, 70, 1] * 5),
    (128, 1, 128, 16, 700, [3, 4, 50]),
    (8, 8, 256, 64, 640, [2, 9] * 20),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,dim,page,shared,lens", DECODES)
def test_decode(dtype, hq, hkv, dim, page, shared, lens):
    """Stale and free parts of the pages hold NaN."""
    c = make_cache(lens, shared, page, hkv, dim, dtype, layers=2, poison=float("nan"))
    tfx.cache_reserve(c, len(lens), hq)
    q = normal((len(lens), hq, dim), dtype, 9, 1.5)
    g = torch.Generator()
    g.manual_seed(3)
    seqs = torch.randperm(len(lens), generator=g).int().cuda()
    check_decode(tfx.attn_decode(c, 1, q, seqs, shared=shared), c, 1, q, seqs)


@pytest.mark.parametrize("shared", [0, 128, 130, 600, 640])
def test_decode_of_uneven_batches(shared):
    """An empty sequence, a slot out of range, one shorter than the shared prefix."""
    lens = [40, 2000, 7, 0]
    c = make_cache(lens, shared, 16, 4, 256, F16, poison=float("inf"))
    if shared:
        c.lens[2] = shared - 60
        c.lens[3] = 0
    tfx.cache_reserve(c, 8, 24)
    q = normal((6, 24, 256), F16, 9)
    seqs = torch.tensor([0, 1, 2, 3, -1, 4], dtype=torch.int32, device="cuda")
    out = tfx.attn_decode(c, 0, q, seqs, shared=shared)
    check_decode(out[:4], c, 0, q[:4], seqs[:4])
    assert not out[4:].any()


@pytest.mark.parametrize("copies", [1, 6])
def test_decode_reads_the_prefix_through_a_sequence_that_holds_it(copies):
    """The batch begins with an empty sequence, a slot out of range and a short one."""
    c = make_cache([5, 9, 70, 33], 400, 16, 4, 256, F16)
    c.lens[0], c.lens[1] = 0, 90
    c.tables[0] = -1
    c.tables[1, 6:] = -1
    tfx.cache_reserve(c, 30, 24)
    seqs = torch.tensor([0, 99, 1, 2, 3] * copies, dtype=torch.int32, device="cuda")
    q = normal((len(seqs), 24, 256), F16, 9)
    out = tfx.attn_decode(c, 0, q, seqs, shared=400)
    keep = [i for i, s in enumerate(seqs.tolist()) if s != 99]
    check_decode(out[keep], c, 0, q[keep], seqs[keep])
    assert not out[1::5].any()


def test_decode_shared_prefix_agrees_with_none():
    c = make_cache([100, 37, 1, 290] * 5, 2000, 16, 4, 256, BF16)
    tfx.cache_reserve(c, 20, 24)
    q = normal((20, 24, 256), BF16, 9)
    seqs = torch.arange(20, dtype=torch.int32, device="cuda")
    a, b = (tfx.attn_decode(c, 0, q, seqs, shared=s, scale=0.09) for s in (2000, 0))
    check_decode(a, c, 0, q, seqs, scale=0.09)
    check_decode(b, c, 0, q, seqs, scale=0.09)
    assert torch.equal(a, tfx.attn_decode(c, 0, q, seqs, shared=2000, scale=0.09))


def test_decode_pitched_on_a_stream_and_in_a_graph():
    c = make_cache([300, 2, 90], 64, 32, 2, 128, F16)
    tfx.cache_reserve(c, 3, 8)
    x = normal((3, 8 * 128 + 24), F16, 4)
    q = x[:, :1024].unflatten(1, (8, 128))
    buf = torch.zeros((3, 8 * 128 + 8), dtype=F16, device="cuda")
    out = buf[:, :1024].unflatten(1, (8, 128))
    seqs = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    tfx.attn_decode(c, 0, q, seqs, shared=64, out=out, stream=st)
    st.synchronize()
    check_decode(out, c, 0, q, seqs)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tfx.attn_decode(c, 0, q, seqs, shared=64, out=out)
    for step in range(3):
        if step == 2:
            c.lens[0] -= 50  # a graph follows the cache's state
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check_decode(out, c, 0, q, seqs)
        assert torch.equal(out, want) == (step < 2)


def test_prompt_in_a_graph():
    q, k, v = normal((200, 6, 256), F16, 1), normal((200, 1, 256), F16, 2), normal((200, 1, 256), F16, 3)
    off, out = offsets_of([150, 50]), torch.empty((200, 6, 256), dtype=F16, device="cuda")
    want = tfx.attn_prompt(q, k, v, off).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tfx.attn_prompt(q, k, v, off, out=out)
    off.zero_()  # the lengths are in the launch, not in this memory
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_bounded_waits_report():
    """With a limit of one cycle every wait gives up on a healthy GPU; the word says so, and the next call is right."""
    q, k, v = normal((300, 6, 256), F16, 1), normal((300, 1, 256), F16, 2), normal((300, 1, 256), F16, 3)
    off = offsets_of([300])
    c = make_cache([300, 2], 640, 32, 2, 128, F16)
    tfx.cache_reserve(c, 2, 8)
    qd, seqs = normal((2, 8, 128), F16, 4), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    want = tfx.attn_prompt(q, k, v, off), tfx.attn_decode(c, 0, qd, seqs, shared=640)
    assert tfx.attn_error() == 0
    tfx.set_spin_limit(1)
    try:
        tfx.attn_prompt(q, k, v, off)
        assert tfx.attn_error() == 1
        tfx.attn_decode(c, 0, qd, seqs, shared=640)
        assert tfx.attn_error() == 1
    finally:
        tfx.set_spin_limit(0)
    assert tfx.attn_error() == 0
    assert torch.equal(tfx.attn_prompt(q, k, v, off), want[0])
    assert torch.equal(tfx.attn_decode(c, 0, qd, seqs, shared=640), want[1])


@pytest.mark.parametrize("hq,hkv,dim,page,shared,lens", [(24, 4, 256, 16, 0, [700, 1, 333]), (8, 2, 128, 16, 200, [90, 2, 1500]),
                                                         (2, 2, 256, 64, 3000, [40] * 8)])
def test_bounded_waits_of_single_warps(hq, hkv, dim, page, shared, lens):
    """Limits at which some lanes' polls succeed and others' do not: a warp gives up as a
    whole, so a call either says that it gave up or is right, and the next call is right."""
    c = make_cache(lens, shared, page, hkv, dim, F16)
    tfx.cache_reserve(c, len(lens), hq)
    q, seqs = normal((len(lens), hq, dim), F16, 4), torch.arange(len(lens), dtype=torch.int32, device="cuda")
    want = tfx.attn_decode(c, 0, q, seqs, shared=shared)
    check_decode(want, c, 0, q, seqs)
    for limit in (1, 300, 700, 1500, 3000):
        tfx.set_spin_limit(limit)
        try:
            got = tfx.attn_decode(c, 0, q, seqs, shared=shared)
            assert tfx.attn_error() == 1 or torch.equal(got, want)
        finally:
            tfx.set_spin_limit(0)
        assert torch.equal(tfx.attn_decode(c, 0, q, seqs, shared=shared), want)
        assert tfx.attn_error() == 0


def test_decode_with_fewer_heads_than_were_reserved():
    """16 sequences of 16 heads take more shares of the prefix than 16 of 24."""
    c = make_cache([5, 40] * 8, 3000, 64, 1, 128, F16)
    tfx.cache_reserve(c, 16, 24)
    seqs = torch.arange(16, dtype=torch.int32, device="cuda")
    for hq, b in ((16, 16), (24, 16), (18, 14), (20, 12), (3, 16), (1, 1)):
        q = normal((b, hq, 128), F16, hq)
        check_decode(tfx.attn_decode(c, 0, q, seqs[:b], shared=3000), c, 0, q, seqs[:b])


@pytest.mark.parametrize("handle", [lambda st: st, lambda st: st.cuda_stream, lambda st: 0], ids=["stream", "handle", "default"])
def test_results_made_for_another_stream(handle):
    """The current stream is far behind: neither the zeros around late sequences nor what it
    still does with memory that it gave back may land in the result."""
    q, k, v = normal((300, 6, 256), F16, 1), normal((300, 1, 256), F16, 2), normal((300, 1, 256), F16, 3)
    off = offsets_of([100, 90], 40)
    c = make_cache([300, 2], 640, 32, 1, 256, F16)
    tfx.cache_reserve(c, 300, 6)
    qd, seqs = normal((300, 6, 256), F16, 4), torch.arange(300, dtype=torch.int32, device="cuda") % 2
    want = tfx.attn_prompt(q, k, v, off), tfx.attn_decode(c, 0, qd, seqs, shared=640)
    torch.cuda.synchronize()
    here, st = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(here):
        for call, w in ((lambda s: tfx.attn_prompt(q, k, v, off, stream=s), want[0]),
                        (lambda s: tfx.attn_decode(c, 0, qd, seqs, shared=640, stream=s), want[1])):
            given_back = torch.empty((300, 6, 256), dtype=F16, device="cuda")
            torch.cuda._sleep(100_000_000)
            given_back.fill_(7.0)
            del given_back
            out = call(handle(st))
            st.synchronize()
            here.synchronize()
            torch.cuda.synchronize()
            assert torch.equal(out, w)
    assert not want[0][:40].any() and not want[0][230:].any()
    check_prompt(want[0], q, k, v, off)


@pytest.mark.parametrize("batch,shared,hq,hkv", [(129, 0, 2, 1), (300, 40, 2, 2), (300, 300, 6, 1), (4096, 0, 1, 1), (4096, 270, 2, 1)])
def test_decode_of_large_batches(batch, shared, hq, hkv):
    """More sequences than one round of the scan over them takes, up to the most that a call takes."""
    lens = [(i * 37) % 61 + (i % 5 > 0) for i in range(batch)]
    c = make_cache(lens, shared, 16, hkv, 128, F16, poison=float("nan"))
    tfx.cache_reserve(c, batch, hq)
    q = normal((batch, hq, 128), F16, 9, 1.5)
    g = torch.Generator()
    g.manual_seed(3)
    seqs = torch.randperm(batch, generator=g).int().cuda()
    out = tfx.attn_decode(c, 0, q, seqs, shared=shared)
    some = list(range(0, batch, max(1, batch // 150))) + [127, 128, batch - 1]
    check_decode(out[some], c, 0, q[some], seqs[some])
    assert torch.isfinite(out).all()
