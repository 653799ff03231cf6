"""Tensors and pools whose elements pass 2^32, and first calls inside a capture."""
import os
import subprocess
import sys

import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx
from test_gpu_attention import check_decode, check_prompt, normal, offsets_of

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GB of free memory are wanted")
    yield
    torch.cuda.empty_cache()


def test_prompts_of_more_than_2_32_elements():
    """q and out of 4.5e9 elements each; the sequences at the ends and around 2^31 and 2^32 elements."""
    n, each, hq, dim = 800, 916, 24, 256
    T = n * each
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q = torch.empty((T, hq, dim), dtype=F16, device="cuda").normal_(0.0, 1.5, generator=g)
    k, v = (torch.empty((T, 2, dim), dtype=F16, device="cuda").normal_(generator=g) for _ in range(2))
    assert q.numel() > 1 << 32
    out = tfx.attn_prompt(q, k, v, offsets_of([each] * n))
    for e in (0, 1 << 31, 1 << 32):
        i = e // (hq * dim * each)
        for s in {i, n - 1}:
            at = slice(s * each, (s + 1) * each)
            check_prompt(out[at], q[at], k[at], v[at], offsets_of([each]), heads=(0, 13, 23))


@pytest.mark.parametrize("dim,page", [(256, 128), (128, 16)])
def test_a_pool_of_more_than_2_32_elements(dim, page):
    """All but the last pages are taken: rows appended, forked, copied and read lie past 2^32 elements, in the second layer."""
    hkv, hq, used = 8, 48, 40
    pages = (1 << 32) // (page * hkv * dim) // 2 + 200
    k, v = (torch.empty((2, pages, page, hkv, dim), dtype=F16, device="cuda") for _ in range(2))
    c = tfx.Cache(k, v, 8, used)
    assert k.numel() > 1 << 32
    tfx.cache_reserve(c, 8, hq)
    c.refs[:pages - used] = 1
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = [20 * page + 3, 1, 5 * page]
    off = offsets_of(lens).cuda()
    tfx.cache_extend(c, ints(0, 1, 2), off)
    kn, vn = normal((sum(lens), hkv, dim), F16, 2), normal((sum(lens), hkv, dim), F16, 3)
    tfx.cache_append(c, 1, kn, vn, ints(0, 1, 2), off)
    tfx.cache_fork(c, ints(0, 1), ints(4, 5))
    assert c.status() == 0 and int(c.tables[0, 0]) == pages - used
    for s, at in ((0, 0), (1, lens[0]), (2, lens[0] + 1), (4, 0), (5, lens[0])):
        n = int(c.lens[s])
        rows = c.tables[s, :-(-n // page)].long()
        for x, new in ((k, kn), (v, vn)):
            assert torch.equal(x[1, rows].reshape(-1, hkv, dim)[:n], new[at:at + n])
    seqs = ints(0, 1, 2, 4, 5)
    q = normal((5, hq, dim), F16, 5, 1.5)
    check_decode(tfx.attn_decode(c, 1, q, seqs), c, 1, q, seqs)
    two = ints(4, 0) if dim == 256 else ints(0, 4)
    q = normal((8, hq, dim), F16, 6, 1.5)
    seqs = two.repeat(4)
    check_decode(tfx.attn_decode(c, 1, q, seqs, shared=lens[0]), c, 1, q, seqs)
    free = (c.refs == 0).nonzero()[:, 0]
    src, dst = c.tables[2, :4].clone(), free[:4].int()
    tfx.cache_copy(c, src, dst)
    for x in (k, v):
        assert torch.equal(x[:, dst.long()], x[:, src.long()])
    # the pool's first pages become free, and everything moves there
    c.refs[:pages - used] = 0
    want = {s: [x[1, c.tables[s, :-(-int(c.lens[s]) // page)].long()].clone() for x in (k, v)] for s in (0, 1, 2, 4, 5)}
    tfx.cache_compact(c)
    assert int(c.book[1]) == int((c.refs > 0).sum()) and int(c.tables.max()) < used
    for s, (wk, wv) in want.items():
        rows = c.tables[s, :-(-int(c.lens[s]) // page)].long()
        assert torch.equal(k[1, rows], wk) and torch.equal(v[1, rows], wv)
    assert c.status() == 0


FIRST = """
import sys, torch
import exl3_trellis_quantized_rot_gb300 as tfx
h = lambda *s: torch.randn(s, device="cuda").half()
q, k, out = h(300, 8, 256), h(300, 2, 256), h(300, 8, 256)
off = torch.tensor([0, 300], dtype=torch.int32)
c = tfx.Cache(h(1, 40, 16, 2, 256), h(1, 40, 16, 2, 256), 4, 30)
tfx.cache_reserve(c, 20, 8)
i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
s, o, b, d, e = i(0), i(0, 300), i(*[0] * 20), i(1), h(20, 8, 256)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    tfx.attn_prompt(q, k, k, off, out=out)
    tfx.cache_extend(c, s, o)
    tfx.cache_append(c, 0, k, k, s, o)
    tfx.cache_append(c, 0, k, k)
    tfx.cache_fork(c, s, d)
    tfx.attn_decode(c, 0, e, b, shared=290, out=e)
    tfx.cache_free(c, d)
    tfx.cache_compact(c)
g.replay()
torch.cuda.synchronize()
assert c.lens.tolist() == [300, 0, 0, 0] and c.status() == 0 and tfx.attn_error() == 0
assert torch.equal(out, tfx.attn_prompt(q, k, k, off)) and torch.isfinite(e).all()
"""


def test_first_calls_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST], check=True, cwd=root, timeout=300)
