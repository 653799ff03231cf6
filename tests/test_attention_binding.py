"""What the attention binding hands to the library, without a GPU: tensors that only say what
they are, and a library that only notes its calls."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import exl3_trellis_quantized_rot_gb300 as tfx  # noqa: E402
from exl3_trellis_quantized_rot_gb300 import attention as at  # noqa: E402

F16, I32 = torch.float16, torch.int32


class Fake:
    """A contiguous CUDA tensor, as far as the binding looks at one."""

    def __init__(self, *shape, dtype=F16, device=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.device = torch.device("cuda", device)

    def stride(self):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s)

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x7F0000000000


class Library:
    """Notes each call by its name; structures by their contents."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name,) + tuple(self.plain(a) for a in args))
            return 0
        return call

    @staticmethod
    def plain(a):
        s = getattr(a, "_obj", None)
        return tuple(getattr(s, f) for f, _ in s._fields_) if isinstance(s, C.Structure) else a


@pytest.fixture
def calls(monkeypatch):
    L = Library()
    monkeypatch.setattr(tfx, "_lib", L)
    if at.torch is None:
        at._load()
    monkeypatch.setattr(at, "_current_device", lambda: 0)
    return L.calls


OFF = torch.tensor([0, 5], dtype=I32)


def entries(device=0):
    """One valid call of every entry point that takes a stream."""
    t = lambda *s, dtype=F16: Fake(*s, dtype=dtype, device=device)  # noqa: E731
    i = lambda n: t(n, dtype=I32)  # noqa: E731
    c = tfx.Cache(t(2, 10, 16, 4, 256), t(2, 10, 16, 4, 256), 3, 5, book=i(4 + 3 + 10 + 15))
    q, k = t(5, 24, 256), t(5, 4, 256)
    return {
        "attn_prompt": lambda **kw: tfx.attn_prompt(q, k, k, OFF, **{"out": q, "stream": 7} | kw),
        "attn_decode": lambda **kw: tfx.attn_decode(c, kw.pop("layer", 0), q, i(5), **{"out": q, "stream": 7} | kw),
        "cache_reserve": lambda b=5, h=24: tfx.cache_reserve(c, b, h, stream=7),
        "cache_extend": lambda: tfx.cache_extend(c, i(2), i(3), stream=7),
        "cache_append": lambda layer=0: tfx.cache_append(c, layer, k, k, stream=7),
        "cache_append_listed": lambda layer=0: tfx.cache_append(c, layer, k, k, i(2), i(3), stream=7),
        "cache_fork": lambda: tfx.cache_fork(c, i(2), i(2), stream=7),
        "cache_free": lambda: tfx.cache_free(c, i(2), stream=7),
        "cache_compact": lambda: tfx.cache_compact(c, stream=7),
        "cache_copy": lambda: tfx.cache_copy(c, i(2), i(2), stream=7),
    }


NAMES = sorted(entries())


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_a_device_that_is_not_the_current_one(calls, name):
    """A launch goes to the current device, whatever the tensors' own."""
    entries()[name]()
    assert [c[0] for c in calls] == ["tfx_" + name]
    with pytest.raises(ValueError, match="current"):
        entries(device=1)[name]()
    assert len(calls) == 1


@pytest.mark.parametrize("name", ["attn_prompt", "attn_decode"])
def test_a_scale_is_taken_by_its_value(calls, name):
    """A tensor that holds the scale may hold another one at the next call."""
    call, scale = entries()[name], torch.tensor(0.25)
    taken = []
    for value in (0.25, 0.5, 0.5):
        scale.fill_(value)
        call(scale=scale)
        taken.append(next(a for a in calls[-1] if isinstance(a, tuple) and len(a) == 5)[4])
    call(scale=2)
    call()
    taken += [next(a for a in c if isinstance(a, tuple) and len(a) == 5)[4] for c in calls[-2:]]
    assert taken == [0.25, 0.5, 0.5, 2.0, 0.0625]


@pytest.mark.parametrize("by", [2 ** 32, -2 ** 32, 2 ** 31])
@pytest.mark.parametrize("name,what", [("attn_decode", dict(shared=5)), ("attn_decode", dict(layer=1)), ("cache_append", dict(layer=1)),
                                       ("cache_append_listed", dict(layer=1)), ("cache_reserve", dict(b=5)),
                                       ("cache_reserve", dict(h=24))])
def test_numbers_past_32_bits_are_refused(calls, name, what, by):
    """The C side would take what is left of them in 32 bits."""
    call = entries()[name]
    call(**what)
    with pytest.raises(ValueError, match="32 bits"):
        call(**{k: v + by for k, v in what.items()})
    assert len(calls) == 1


def test_a_cache_in_host_memory_is_refused(calls):
    """Its lists would be host tensors too, and the kernels would be given their addresses."""
    k = torch.zeros(1, 2, 16, 1, 128, dtype=F16)
    with pytest.raises(ValueError, match="CUDA"):
        c = tfx.Cache(k, k.clone(), 1, 2)
        tfx.cache_extend(c, torch.zeros(1, dtype=I32), torch.zeros(2, dtype=I32), stream=7)
