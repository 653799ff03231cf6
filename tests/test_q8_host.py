"""Refusals of the 8-bit cache's and the rotary calls, without a GPU, and the rotary table."""
import ctypes as C
import math
import os
import re
from fractions import Fraction

import pytest

import exl3_trellis_quantized_rot_gb300 as tfx
from exl3_trellis_quantized_rot_gb300 import attention as at
from exl3_trellis_quantized_rot_gb300 import rotary

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


def cache(**kw):
    d = dict(k=P, v=P, book=P, layers=2, pages=10, page_size=16, heads_kv=4, dim=256, act=0, slots=3, width=5, priv=None,
             store=at.STORE_I8, k_scale=P, v_scale=P)
    return at.CacheStruct(*(d | kw).values())


def test_every_declared_symbol_is_exported(L):
    src = open(os.path.join(ROOT, "include", "tfx_rope.h")).read()
    names = set(re.findall(r"^int (tfx_[a-z_]+)\(", src, re.M))
    assert names == set(rotary.ABI_SYMBOLS) and all(hasattr(L, n) for n in names)


@pytest.mark.parametrize("kw,code", [
    (dict(store=3), tfx.EINVAL), (dict(store=-1), tfx.EINVAL), (dict(k_scale=None), tfx.EINVAL), (dict(v_scale=None), tfx.EINVAL),
    (dict(k_scale=P + 2), tfx.EALIGN), (dict(v_scale=P + 1), tfx.EALIGN), (dict(act=2), tfx.EINVAL), (dict(dim=64), tfx.EUNSUPPORTED),
    (dict(page_size=8), tfx.EUNSUPPORTED)])
def test_cache_refusals(L, drv, kw, code):
    c = cache(**kw)
    r = C.byref(c)
    h = C.byref(at.HeadsStruct(24, 4, 256, 0, 0.0625))
    assert L.tfx_cache_reserve(r, 1, 24, None) == code
    assert L.tfx_cache_append(r, 0, P, 1024, P, 1024, 1, None) == code
    assert L.tfx_cache_read(r, 0, P, P, P, 1, 1, P, 1024, P, 1024, None) == code
    assert L.tfx_attn_decode(r, 0, h, P, 6144, P, 1, 0, P, 6144, None) == code
    assert not drv.live and tfx.last_error()


@pytest.mark.parametrize("store", [at.STORE_ACT, at.STORE_I8, at.STORE_E4M3])
def test_read_refusals(L, drv, store):
    c = cache(store=store)
    r = C.byref(c)
    read = lambda layer=0, seqs=P, starts=P, off=P, n=1, rows=1, k=P, ldk=1024, v=P, ldv=1024: L.tfx_cache_read(  # noqa: E731
        r, layer, seqs, starts, off, n, rows, k, ldk, v, ldv, None)
    assert read() == tfx.ENOTRESERVED
    assert L.tfx_cache_reserve(r, 1, 24, None) == 0
    assert read(layer=-1) == tfx.EINVAL and read(layer=2) == tfx.EINVAL and read(n=-1) == tfx.EINVAL and read(rows=-1) == tfx.EINVAL
    assert read(seqs=None) == tfx.EINVAL and read(starts=None) == tfx.EINVAL and read(off=None) == tfx.EINVAL
    assert read(k=None) == tfx.EINVAL and read(v=None) == tfx.EINVAL and read(ldk=1016) == tfx.EINVAL
    assert read(k=P + 8) == tfx.EALIGN and read(ldv=1028) == tfx.EALIGN and read(k=P, v=P) == tfx.EINVAL
    n = tfx.launch_count()
    assert read(n=0, seqs=None, starts=None, off=None) == 0 and read(rows=0, k=None, v=None) == 0
    assert tfx.launch_count() == n
    assert L.tfx_cache_release(r) == 0


def test_a_reservation_grows_with_heads_and_sequences(L, drv):
    def taken(batch, hq):
        c = cache()
        assert L.tfx_cache_reserve(C.byref(c), batch, hq, None) == 0
        n = sum(drv.live.values())
        assert L.tfx_cache_release(C.byref(c)) == 0
        return n

    size = {(b, g): taken(b, 4 * g) for b in (1, 2, 3, 17, 64, 900) for g in (1, 2, 6, 16, 20, 128)}
    for (b, g), n in size.items():
        assert all(m <= n for (x, y), m in size.items() if x <= b and y <= g)


def test_a_reservation_for_two_sequences_has_no_room_for_the_prefix_s_kernel(L, drv):
    """Batches of one and two read a prefix as their own: 128 rows of FP32 an SM less than a batch of three takes."""
    def taken(batch):
        c = cache(heads_kv=1)
        assert L.tfx_cache_reserve(C.byref(c), batch, 1, None) == 0
        n = sum(drv.live.values())
        assert L.tfx_cache_release(C.byref(c)) == 0
        return n

    one, two, three = taken(1), taken(2), taken(3)
    assert one <= two < three
    assert three - two >= 128 * 256 * 4 * 100  # GB300 has 152 SMs
    c = cache(heads_kv=1)
    r = C.byref(c)
    assert L.tfx_cache_reserve(r, 2, 1, None) == 0
    h = C.byref(at.HeadsStruct(1, 1, 256, 0, 0.0625))
    assert L.tfx_attn_decode(r, 0, h, P, 256, P, 3, 80, P, 256, None) == tfx.ENOTRESERVED
    assert L.tfx_cache_reserve(r, 3, 1, None) == 0  # it grows
    assert L.tfx_cache_release(r) == 0 and not drv.live


@pytest.mark.parametrize("store", [at.STORE_ACT, at.STORE_I8, at.STORE_E4M3])
@pytest.mark.parametrize("heads,dim", [(1 << 23, 256), ((1 << 22) + 1, 256), (1 << 24, 128), (1 << 27, 128)])
def test_tokens_of_more_values_than_the_kernels_count(L, drv, store, heads, dim):
    """heads_kv * dim is a 32-bit number in the append, read and copy kernels."""
    c = cache(store=store, heads_kv=heads, dim=dim)
    r = C.byref(c)
    assert L.tfx_cache_reserve(r, 1, heads, None) == tfx.EUNSUPPORTED and "2^30" in tfx.last_error()
    assert L.tfx_cache_append(r, 0, P, heads * dim, P, heads * dim, 1, None) == tfx.EUNSUPPORTED
    assert L.tfx_cache_read(r, 0, P, P, P, 1, 1, P, heads * dim, P, heads * dim, None) == tfx.EUNSUPPORTED
    assert not drv.live


def rope_args(**kw):
    d = dict(act=0, dim=128, q=P, ldq=512, heads_q=4, q_out=P + (1 << 30), ldqo=512, k=P + (1 << 31), ldk=256, heads_k=2,
             k_out=P + (1 << 32), ldko=256, positions=P, rows=3, inverse=0, stream=None)
    assert set(kw) <= set(d)
    return tuple((d | kw).values())


@pytest.mark.parametrize("kw,code", [
    (dict(act=2), tfx.EINVAL), (dict(dim=8), tfx.EINVAL), (dict(dim=132), tfx.EALIGN), (dict(dim=32), tfx.EUNSUPPORTED),
    (dict(heads_q=0), tfx.EINVAL), (dict(heads_k=-1), tfx.EINVAL), (dict(heads_q=70000), tfx.EINVAL), (dict(rows=-1), tfx.EINVAL),
    (dict(q=None), tfx.EINVAL), (dict(q_out=None), tfx.EINVAL), (dict(k=None), tfx.EINVAL), (dict(k_out=None), tfx.EINVAL),
    (dict(positions=None), tfx.EINVAL), (dict(positions=P + 2), tfx.EALIGN), (dict(ldq=504), tfx.EINVAL), (dict(ldqo=508), tfx.EINVAL),
    (dict(ldk=260), tfx.EALIGN), (dict(ldko=1 << 37), tfx.EINVAL), (dict(q=P + 8), tfx.EALIGN), (dict(k_out=P + 4), tfx.EALIGN),
    (dict(q_out=P, ldqo=520), tfx.EINVAL)])
def test_rope_refusals(L, kw, code):
    r = rotary.RopeStruct(P, 64, 0, 1.0)
    n = tfx.launch_count()
    assert L.tfx_rope_apply(C.byref(r), *rope_args(**kw)) == code
    assert tfx.last_error() and tfx.launch_count() == n


@pytest.mark.parametrize("kw", [dict(q_out=P + (1 << 31)), dict(k_out=P), dict(k_out=P + (1 << 30))])
def test_rope_outputs_that_are_other_tensors(L, kw):
    r = rotary.RopeStruct(P, 64, 0, 1.0)
    n = tfx.launch_count()
    assert L.tfx_rope_apply(C.byref(r), *rope_args(**kw)) == tfx.EINVAL
    assert "output" in tfx.last_error() and tfx.launch_count() == n


@pytest.mark.parametrize("table,rotary_dim,gain,code", [
    (None, 64, 1.0, tfx.EINVAL), (P + 4, 64, 1.0, tfx.EALIGN), (P, 0, 1.0, tfx.EUNSUPPORTED), (P, 24, 1.0, tfx.EUNSUPPORTED),
    (P, 144, 1.0, tfx.EUNSUPPORTED), (P, 64, float("nan"), tfx.EINVAL)])
def test_rope_plan_refusals(L, table, rotary_dim, gain, code):
    r = rotary.RopeStruct(table, rotary_dim, 0, gain)
    assert L.tfx_rope_apply(C.byref(r), *rope_args()) == code


def test_no_rows_is_no_error(L):
    r = rotary.RopeStruct(P, 64, 0, 1.0)
    n = tfx.launch_count()
    assert L.tfx_rope_apply(C.byref(r), *rope_args(rows=0, q=None, k=None, positions=None)) == 0
    assert tfx.launch_count() == n


def test_rope_table(L):
    """Fractions of a turn: within 2^-51 of the frequency over 2 pi, and of 2^-64."""
    f = [1.0, 0.5, 1e-7, 0.0, -1.0, 7.0, -1e-30, 2 * math.pi, 123456.789, 10000 ** (-2 * 5 / 128)]
    t = (C.c_uint64 * len(f))()
    assert L.tfx_rope_table((C.c_double * len(f))(*f), len(f), t) == 0
    pi = Fraction(3141592653589793238462643383279502884197, 10 ** 39)
    for x, n in zip(f, t):
        turns = Fraction(x) / (2 * pi)
        off = (turns - Fraction(n, 2 ** 64)) % 1
        off = min(off, 1 - off)
        assert off <= abs(turns) * Fraction(1, 2 ** 51) + Fraction(1, 2 ** 53)
    assert L.tfx_rope_table((C.c_double * 2)(1.0, float("inf")), 2, t) == tfx.EINVAL
    assert L.tfx_rope_table(None, 1, t) == tfx.EINVAL and L.tfx_rope_table(None, 0, None) == 0 and L.tfx_rope_table(None, -1, None) == tfx.EINVAL


def test_frequencies():
    f, gain = tfx.rope_frequencies(64, 10000.0)
    assert gain == 1.0 and f[0] == 1.0 and all(abs(x - 10000 ** (-2 * i / 64)) <= 1e-15 for i, x in enumerate(f))
    g, _ = tfx.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert g == [x / 4 for x in f]
    g, _ = tfx.rope_frequencies(64, 10000.0, "ntk", 4.0)
    assert g[0] == 1.0 and abs(g[-1] / f[-1] - 1 / 4) < 1e-12  # the slowest pair reaches as far as `factor` times the context
    g, gain = tfx.rope_frequencies(64, 10000.0, "yarn", 4.0, original=4096)
    assert abs(gain - (0.1 * math.log(4) + 1)) < 1e-15
    ratio = [a / b for a, b in zip(g, f)]
    assert ratio[0] == 1.0 and abs(ratio[-1] - 0.25) < 1e-12 and all(a >= b for a, b in zip(ratio, ratio[1:]))
    turns = [4096 * x / (2 * math.pi) for x in f]
    assert all(r == 1.0 for r, t in zip(ratio, turns) if t > 50) and all(abs(r - 0.25) < 1e-12 for r, t in zip(ratio, turns) if t < 0.7)
    for kw in (dict(scaling="dynamic"), dict(base=1.0), dict(factor=0.0), dict(slow=32.0, fast=1.0), dict(original=0)):
        with pytest.raises(ValueError):
            tfx.rope_frequencies(64, **({"scaling": "yarn"} | kw))
    for r in (3, 2, 0):
        with pytest.raises(ValueError):
            tfx.rope_frequencies(r)


def test_binding_refuses_wrong_tensors(monkeypatch):
    torch = pytest.importorskip("torch")
    if at.torch is None:
        at._load()
    monkeypatch.setattr(at, "_current_device", lambda: 0)
    k8 = torch.zeros(1, 4, 32, 2, 128, dtype=torch.int8)
    k16 = torch.zeros(1, 4, 32, 2, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="act"):
        tfx.Cache(k8, k8.clone(), 1, 2)
    with pytest.raises(ValueError, match="dtype"):
        tfx.Cache(k8, k8.clone(), 1, 2, act=torch.float32)
    with pytest.raises(ValueError, match="act and scales"):
        tfx.Cache(k16, k16.clone(), 1, 2, act=torch.bfloat16)
    with pytest.raises(ValueError, match="act and scales"):
        tfx.Cache(k16, k16.clone(), 1, 2, k_scale=torch.zeros(1, 4, 2, 2))
    with pytest.raises(ValueError, match="one shape, type"):
        tfx.Cache(k8, k8.view(torch.float8_e4m3fn), 1, 2, act=torch.float16)
    for bad in (torch.zeros(1, 4, 1, 2), torch.zeros(1, 4, 2, 2, dtype=torch.float64), torch.zeros(1, 4, 2, 4)[..., ::2]):
        with pytest.raises(ValueError, match="v_scale"):
            tfx.Cache(k8, k8.clone(), 1, 2, act=torch.float16, v_scale=bad)
    c = tfx.Cache(k8, k8.clone(), 1, 2, act=torch.bfloat16)
    assert c.k_scale.shape == (1, 4, 2, 2) and c.s.store == at.STORE_I8 and c.dtype == torch.bfloat16
    ints = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tfx.cache_read(c, 0, ints, ints, torch.zeros(2, dtype=torch.int32), 1, stream=7)
    for kw in (dict(rotary=24), dict(rotary=0), dict(rotary=144), dict(freqs=[1.0] * 3), dict(freqs=[1.0] * 64, scaling="ntk")):
        with pytest.raises(ValueError):
            tfx.Rope(128, **kw, device="cpu")
    with pytest.raises(ValueError, match="multiple"):
        tfx.Rope(132, rotary=32, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        tfx.Rope(128, device="cpu")
