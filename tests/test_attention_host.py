"""Refusals of the attention and cache calls, without a GPU: each is checked before any CUDA call."""
import ctypes as C
import os
import re

import pytest

import exl3_trellis_quantized_rot_gb300 as tfx
from exl3_trellis_quantized_rot_gb300 import attention as at

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x7F0000000000  # an aligned stand-in address, never read on the host


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build_library()
    return tfx.lib()


class FakeDriver:
    def __init__(self):
        self.live, self.next = {}, 1 << 20
        self.s = tfx.DriverStruct(tfx.ALLOC_FN(self._alloc), tfx.FREE_FN(self._free), tfx.MEMSET_FN(lambda p, n, s: 0))

    def _alloc(self, pp, n, s):
        pp[0] = self.next
        self.live[self.next] = n
        self.next += n + 4096
        return 0

    def _free(self, p, s):
        del self.live[p]
        return 0


@pytest.fixture
def drv(L):
    d = FakeDriver()
    tfx.set_driver(d.s)
    yield d
    tfx.set_driver(None)


def heads(hq=24, hkv=4, dim=256, act=0, scale=0.0625):
    return at.HeadsStruct(hq, hkv, dim, act, scale)


def cache(**kw):
    d = dict(k=P, v=P, book=P, layers=2, pages=10, page_size=16, heads_kv=4, dim=256, act=0, slots=3, width=5, priv=None)
    return at.CacheStruct(*(d | kw).values())


def prompt(L, h=None, q=P, ldq=6144, k=P, ldk=1024, v=P, ldv=1024, offsets=(0, 5), n=None, out=P, ldo=6144):
    o = (C.c_int32 * len(offsets))(*offsets) if offsets is not None else None
    return L.tfx_attn_prompt(C.byref(h or heads()), q, ldq, k, ldk, v, ldv, o, len(offsets) - 1 if n is None else n, out, ldo,
                             None)


def test_every_declared_symbol_is_exported(L):
    src = open(os.path.join(ROOT, "include", "tfx_attn.h")).read()
    names = set(re.findall(r"^int(?:64_t)? (tfx_[a-z_]+)\(", src, re.M))
    assert names == set(at.ABI_SYMBOLS)
    for n in names:
        assert hasattr(L, n), n


@pytest.mark.parametrize("kw,code", [
    (dict(h=heads(hq=25)), tfx.EINVAL), (dict(h=heads(hq=0)), tfx.EINVAL), (dict(h=heads(hkv=0)), tfx.EINVAL),
    (dict(h=heads(hq=258, hkv=2)), tfx.EINVAL), (dict(h=heads(dim=64)), tfx.EUNSUPPORTED), (dict(h=heads(act=2)), tfx.EINVAL),
    (dict(h=heads(scale=0.0)), tfx.EINVAL), (dict(h=heads(scale=float("nan"))), tfx.EINVAL),
    (dict(h=heads(scale=float("inf"))), tfx.EINVAL), (dict(n=-1), tfx.EINVAL), (dict(offsets=None, n=2), tfx.EINVAL),
    (dict(offsets=(-1, 4)), tfx.EINVAL), (dict(offsets=(0, 4, 3)), tfx.EINVAL), (dict(q=None), tfx.EINVAL),
    (dict(k=None), tfx.EINVAL), (dict(v=None), tfx.EINVAL), (dict(out=None), tfx.EINVAL), (dict(q=P + 8), tfx.EALIGN),
    (dict(v=P + 2), tfx.EALIGN), (dict(ldq=6143), tfx.EINVAL), (dict(ldq=6148), tfx.EALIGN), (dict(ldk=1020), tfx.EINVAL),
    (dict(ldo=6150), tfx.EALIGN)])
def test_prompt_refusals(L, kw, code):
    assert prompt(L, **kw) == code
    assert tfx.last_error()


def test_nothing_to_do_is_no_error(L):
    n = tfx.launch_count()
    assert prompt(L, offsets=(0,)) == 0 and prompt(L, offsets=(7, 7, 7), q=None) == 0
    assert tfx.launch_count() == n


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), tfx.EINVAL), (dict(book=None), tfx.EINVAL), (dict(layers=0), tfx.EINVAL), (dict(pages=0), tfx.EINVAL),
    (dict(slots=0), tfx.EINVAL), (dict(width=0), tfx.EINVAL), (dict(heads_kv=0), tfx.EINVAL), (dict(act=5), tfx.EINVAL),
    (dict(dim=96), tfx.EUNSUPPORTED), (dict(page_size=24), tfx.EUNSUPPORTED), (dict(page_size=256), tfx.EUNSUPPORTED),
    (dict(pages=1 << 28), tfx.EUNSUPPORTED), (dict(v=P + 8), tfx.EALIGN), (dict(book=P + 2), tfx.EALIGN)])
def test_cache_refusals(L, drv, kw, code):
    c = cache(**kw)
    r = C.byref(c)
    assert L.tfx_cache_reserve(r, 1, 24, None) == code
    assert L.tfx_cache_extend(r, P, P, 1, None) == code
    assert L.tfx_cache_append(r, 0, P, 1024, P, 1024, 1, None) == code
    assert L.tfx_cache_compact(r, None) == code
    assert L.tfx_attn_decode(r, 0, C.byref(heads()), P, 6144, P, 1, 0, P, 6144, None) == code
    assert not drv.live


def test_calls_refuse_before_reserve_and_past_it(L, drv):
    c = cache()
    r, h = C.byref(c), heads()
    dec = lambda layer=0, hh=h, q=P, ldq=6144, seqs=P, batch=2, shared=0, out=P, ldo=6144: L.tfx_attn_decode(  # noqa: E731
        r, layer, C.byref(hh), q, ldq, seqs, batch, shared, out, ldo, None)
    for rc in (L.tfx_cache_extend(r, P, P, 1, None), L.tfx_cache_append(r, 0, P, 1024, P, 1024, 1, None),
               L.tfx_cache_fork(r, P, P, 1, None), L.tfx_cache_free(r, P, 1, None), L.tfx_cache_compact(r, None),
               L.tfx_cache_copy(r, P, P, 1, None), dec()):
        assert rc == tfx.ENOTRESERVED
    for b, hq in ((0, 24), (at.MAX_BATCH + 1, 24), (1, 0), (1, 25), (1, 4 * 129)):
        assert L.tfx_cache_reserve(r, b, hq, None) == tfx.EINVAL
    assert L.tfx_cache_reserve(r, 2, 24, None) == 0
    held = dict(drv.live)
    assert L.tfx_cache_reserve(r, 1, 24, None) == 0 and drv.live == held  # grow only
    assert dec(batch=3) == tfx.ENOTRESERVED
    assert dec(hh=heads(hq=48), ldq=12288, ldo=12288) == tfx.ENOTRESERVED
    assert dec(hh=heads(hkv=8)) == tfx.EINVAL and dec(hh=heads(dim=128)) == tfx.EINVAL and dec(hh=heads(act=1)) == tfx.EINVAL
    assert dec(layer=2) == tfx.EINVAL and dec(layer=-1) == tfx.EINVAL and dec(batch=-1) == tfx.EINVAL
    assert dec(shared=-1) == tfx.EINVAL and dec(shared=81) == tfx.EINVAL
    assert dec(q=None) == tfx.EINVAL and dec(seqs=None) == tfx.EINVAL and dec(out=None) == tfx.EINVAL
    assert dec(q=P + 4) == tfx.EALIGN and dec(ldo=6145) == tfx.EALIGN and dec(ldq=6140) == tfx.EINVAL
    assert dec(batch=0) == 0
    assert L.tfx_cache_extend(r, P, P, 4, None) == tfx.EINVAL and L.tfx_cache_extend(r, None, P, 1, None) == tfx.EINVAL
    assert L.tfx_cache_fork(r, P, None, 1, None) == tfx.EINVAL and L.tfx_cache_fork(r, P, P, -1, None) == tfx.EINVAL
    assert L.tfx_cache_free(r, None, 1, None) == tfx.EINVAL and L.tfx_cache_copy(r, P, P, 11, None) == tfx.EINVAL
    assert L.tfx_cache_append(r, 2, P, 1024, P, 1024, 1, None) == tfx.EINVAL
    assert L.tfx_cache_append(r, 0, P, 1024, P, 1024, 161, None) == tfx.EINVAL
    assert L.tfx_cache_append(r, 0, P, 1023, P, 1024, 1, None) == tfx.EINVAL
    assert L.tfx_cache_append(r, 0, P, 1024, P, 1028, 1, None) == tfx.EALIGN
    assert L.tfx_cache_append(r, 0, P, 1024, P, 1024, 0, None) == 0
    assert L.tfx_cache_fork(r, P, P, 0, None) == 0 and L.tfx_cache_free(r, None, 0, None) == 0
    assert L.tfx_cache_release(r) == 0 and not drv.live and c.priv is None
    assert L.tfx_cache_release(r) == 0


def test_book_size(L):
    assert L.tfx_cache_book_ints(C.byref(cache())) == 4 + 3 + 10 + 15
    assert L.tfx_cache_book_ints(None) == 0


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(4, 6, 256, dtype=torch.float16), torch.zeros(4, 1, 256, dtype=torch.float16)
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tfx.attn_prompt(q, k, k, off)
    with pytest.raises(ValueError, match="rows, heads, dim"):
        tfx.attn_prompt(q[0], k, k, off)
    with pytest.raises(ValueError, match="contiguous"):
        tfx.Cache(torch.zeros(1, 2, 16, 4, 128).half()[:, :, :, ::2], torch.zeros(1, 2, 16, 4, 128).half()[:, :, :, ::2], 1, 1)
    with pytest.raises(ValueError, match="dtype"):
        tfx.Cache(torch.zeros(1, 2, 16, 2, 128), torch.zeros(1, 2, 16, 2, 128), 1, 1)
    with pytest.raises(ValueError, match="book"):
        tfx.Cache(k.view(1, 1, 4, 1, 256), k.view(1, 1, 4, 1, 256), 1, 1, book=torch.zeros(3, dtype=torch.int32))


def test_append_with_lists_refusals(L, drv):
    c = cache()
    r = C.byref(c)
    app = lambda layer=0, k=P, ldk=1024, rows=1, seqs=P, off=P, n=1: L.tfx_cache_append_listed(  # noqa: E731
        r, layer, k, ldk, P, 1024, rows, seqs, off, n, None)
    assert app() == tfx.ENOTRESERVED
    assert L.tfx_cache_reserve(r, 2, 24, None) == 0
    assert app(n=-1) == tfx.EINVAL and app(n=4) == tfx.EINVAL and app(seqs=None) == tfx.EINVAL and app(off=None) == tfx.EINVAL
    assert app(layer=2) == tfx.EINVAL and app(rows=-1) == tfx.EINVAL and app(rows=161) == tfx.EINVAL
    assert app(k=None) == tfx.EINVAL and app(ldk=1028) == tfx.EALIGN
    n = tfx.launch_count()
    assert app(rows=0) == 0 and app(n=0, seqs=None, off=None) == 0 and tfx.launch_count() == n
    assert L.tfx_cache_release(r) == 0


def test_a_reservation_that_cannot_clear_its_scratch_holds_nothing(L, drv):
    drv.s.memset0 = tfx.MEMSET_FN(lambda p, n, s: -1)
    tfx.set_driver(drv.s)
    c = cache()
    r = C.byref(c)
    assert L.tfx_cache_reserve(r, 2, 24, None) == tfx.ECUDA and not drv.live
    assert L.tfx_cache_extend(r, P, P, 1, None) == tfx.ENOTRESERVED
    assert L.tfx_cache_release(r) == 0


@pytest.mark.parametrize("hkv", [1, 4])
def test_a_reservation_holds_for_fewer_heads_and_sequences(L, drv, hkv):
    """What it takes does not shrink with batch or heads: a call within both finds its room."""
    def taken(batch, group):
        c = cache(heads_kv=hkv)
        assert L.tfx_cache_reserve(C.byref(c), batch, group * hkv, None) == 0
        n = sum(drv.live.values())
        assert L.tfx_cache_release(C.byref(c)) == 0
        return n

    batches, groups = (1, 2, 5, 12, 14, 16, 21, 28, 32, 64, 200), (1, 2, 3, 4, 6, 8, 11, 16, 18, 20, 21, 24, 32, 64, 100, 128)
    size = {(b, g): taken(b, g) for b in batches for g in groups}
    for b in batches:
        for g in groups:
            assert all(size[x, y] <= size[b, g] for x in batches for y in groups if x <= b and y <= g), (b, g)


@pytest.mark.parametrize("kw", [dict(width=(1 << 27) - 1), dict(width=(1 << 24) - 1, page_size=128), dict(width=(1 << 27) - 127),
                                dict(slots=1 << 16, width=1 << 16), dict(slots=1 << 20, width=(1 << 11) + 1)])
def test_sizes_whose_positions_or_entries_pass_32_bits(L, drv, kw):
    """Kernels count tokens a sequence (and look a thousand ahead) and table entries in 32 bits."""
    assert L.tfx_cache_reserve(C.byref(cache(**kw)), 1, 24, None) == tfx.EUNSUPPORTED and not drv.live


@pytest.mark.parametrize("kw", [dict(width=(1 << 27) - 128), dict(slots=1 << 16, width=(1 << 15) - 1)])
def test_the_largest_sizes(L, drv, kw):
    c = cache(**kw)
    assert L.tfx_cache_reserve(C.byref(c), 1, 24, None) == 0
    assert L.tfx_cache_release(C.byref(c)) == 0


def test_decode_of_more_slices_than_are_counted_in_32_bits(L, drv):
    """A step's own tokens are numbered through in slices of 16 (dim 256) or 32 keys."""
    c = cache(width=1 << 22, page_size=128, slots=128)  # 2^29 tokens a sequence
    r = C.byref(c)
    assert L.tfx_cache_reserve(r, 128, 24, None) == 0
    dec = lambda batch, hh: L.tfx_attn_decode(r, 0, C.byref(hh), P, 6144, P, batch, 0, P, 6144, None)  # noqa: E731
    assert dec(64, heads()) == tfx.EUNSUPPORTED and dec(128, heads()) == tfx.EUNSUPPORTED
    assert dec(63, heads()) != tfx.EUNSUPPORTED
    assert L.tfx_cache_release(r) == 0
