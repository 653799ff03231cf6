"""What the binding of rotary positions and of the 8-bit cache hands to the library, without a GPU."""
import pytest

torch = pytest.importorskip("torch")

import exl3_trellis_quantized_rot_gb300 as tfx  # noqa: E402
from exl3_trellis_quantized_rot_gb300 import attention as at, rotary  # noqa: E402
from test_attention_binding import Fake, calls  # noqa: E402, F401

F16, BF16, I8, I32, F32 = torch.float16, torch.bfloat16, torch.int8, torch.int32, torch.float32


def entries(device=0, act=BF16):
    t = lambda *s, dtype=act: Fake(*s, dtype=dtype, device=device)  # noqa: E731
    i = lambda n: t(n, dtype=I32)  # noqa: E731
    c = tfx.Cache(t(2, 10, 32, 4, 256, dtype=I8), t(2, 10, 32, 4, 256, dtype=I8), 3, 5, book=i(4 + 3 + 10 + 15),
                  k_scale=t(2, 10, 2, 4, dtype=F32), v_scale=t(2, 10, 2, 4, dtype=F32), act=act)
    r = tfx.Rope.__new__(tfx.Rope)  # its table would be a copy to a GPU
    r.dim, r.rotary, r.device, r.s = 256, 64, device, rotary.RopeStruct(0x7F0000000000, 64, 0, 1.0)
    r.ref = rotary.C.byref(r.s)
    q, k = t(5, 24, 256), t(5, 4, 256)
    return {
        "rope_apply": lambda **kw: tfx.rope(r, q, k, i(5), **{"out": (q, k), "stream": 7} | kw),
        "cache_read": lambda layer=1, rows=5, **kw: tfx.cache_read(c, layer, i(2), i(2), i(3), rows, **{"out": (k, k), "stream": 7} | kw),
        "cache_append": lambda layer=1: tfx.cache_append(c, layer, k, k, stream=7),
        "attn_decode": lambda **kw: tfx.attn_decode(c, kw.pop("layer", 0), q, i(5), **{"out": q, "stream": 7} | kw),
    }


@pytest.mark.parametrize("name", sorted(entries()))
def test_tensors_of_a_device_that_is_not_the_current_one(calls, name):  # noqa: F811
    entries()[name]()
    assert [c[0] for c in calls] == ["tfx_" + name]
    with pytest.raises(ValueError, match="current"):
        entries(device=1)[name]()
    assert len(calls) == 1


@pytest.mark.parametrize("name", ["cache_read", "cache_append"])
def test_the_cache_s_types_reach_the_library(calls, name):  # noqa: F811
    entries(act=BF16)[name]()
    s = dict(zip((f for f, _ in at.CacheStruct._fields_), calls[-1][1]))
    assert s["act"] == 1 and s["store"] == at.STORE_I8 and s["k_scale"] and s["v_scale"] and calls[-1][2] == 1


@pytest.mark.parametrize("by", [2 ** 32, -2 ** 32, 2 ** 31])
@pytest.mark.parametrize("what", [dict(layer=1), dict(rows=5)])
def test_numbers_past_32_bits_are_refused(calls, what, by):  # noqa: F811
    with pytest.raises(ValueError, match="32 bits"):
        entries()["cache_read"](**{k: v + by for k, v in what.items()})
    assert not calls


def test_shapes_types_and_devices_that_do_not_go_together(calls):  # noqa: F811
    t = Fake
    e = entries(act=F16)
    for out in ((t(5, 24, 256), None), (t(4, 24, 256), t(5, 4, 256)), (t(5, 24, 256), t(6, 4, 256)),
                (t(5, 24, 256, dtype=BF16), t(5, 4, 256)), (t(5, 24, 256, device=1), t(5, 4, 256)), (t(5, 24, 128), t(5, 4, 256))):
        with pytest.raises(ValueError):
            e["rope_apply"](out=out)
    for out in ((t(4, 4, 256), t(5, 4, 256)), (t(5, 4, 256), t(5, 4, 256, dtype=BF16)), (t(5, 4, 256), t(5, 4, 256, device=1)),
                (t(5, 2, 256), t(5, 4, 256))):
        with pytest.raises(ValueError):
            e["cache_read"](out=out)
    with pytest.raises(ValueError):
        e["cache_read"](rows=-1)
    assert not calls
    e["cache_read"](out=(t(9, 4, 256), t(7, 4, 256)))  # more rows than are read
    assert len(calls) == 1


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 2])
def test_lists_past_32_bits_are_refused(calls, n):  # noqa: F811
    """Modulo 2^32 the library would see a few of their entries, or none."""
    i = lambda n: Fake(n, dtype=I32)  # noqa: E731
    t = lambda *s, dtype=F16: Fake(*s, dtype=dtype)  # noqa: E731
    c = tfx.Cache(t(2, 10, 32, 4, 256), t(2, 10, 32, 4, 256), 3, 5, book=i(4 + 3 + 10 + 15))
    k = t(5, 4, 256)
    r = tfx.Rope.__new__(tfx.Rope)
    r.dim, r.rotary, r.device, r.s = 16, 16, 0, rotary.RopeStruct(0x7F0000000000, 16, 0, 1.0)
    r.ref = rotary.C.byref(r.s)
    x = t(n, 1, 16)
    for call in (lambda: tfx.cache_read(c, 0, i(n), i(n), i(n + 1), 5, out=(k, k), stream=7),
                 lambda: tfx.cache_extend(c, i(n), i(n + 1), stream=7),
                 lambda: tfx.cache_append(c, 0, k, k, i(n), i(n + 1), stream=7),
                 lambda: tfx.cache_fork(c, i(n), i(n), stream=7), lambda: tfx.cache_copy(c, i(n), i(n), stream=7),
                 lambda: tfx.cache_free(c, i(n), stream=7), lambda: tfx.rope(r, x, x, i(n), out=(x, x), stream=7)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert not calls


@pytest.mark.parametrize("heads,kv", [(2 ** 32 + 24, 1), (1, 2 ** 32), (2 ** 31, 0)])
def test_rotated_heads_past_32_bits_are_refused(calls, heads, kv):  # noqa: F811
    """Modulo 2^32 the library would see a few of them and leave the rest as they are."""
    r = tfx.Rope.__new__(tfx.Rope)
    r.dim, r.rotary, r.device, r.s = 16, 16, 0, rotary.RopeStruct(0x7F0000000000, 16, 0, 1.0)
    r.ref = rotary.C.byref(r.s)
    q, k = Fake(2, heads, 16), Fake(2, kv, 16) if kv else None
    with pytest.raises(ValueError, match="32 bits"):
        tfx.rope(r, q, k, Fake(2, dtype=I32), out=(q, k), stream=7)
    assert not calls
