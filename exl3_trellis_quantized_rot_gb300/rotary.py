"""Python binding of the tfx_rope C ABI: rotary positions.

Argument marshalling and shape checks only, as in the package's other parts: rows are
rotated by the kernels of ``libtfx_exl3.so``. ``Rope`` is the plan (frequencies of a model,
made once), ``rope`` the call.
"""
from __future__ import annotations

import ctypes as C
import math

from . import attention as _at

ABI_SYMBOLS = ("tfx_rope_table", "tfx_rope_apply")


class RopeStruct(C.Structure):
    _fields_ = [("table", C.c_void_p), ("rotary", C.c_int), ("interleaved", C.c_int), ("gain", C.c_float)]


def declare(L: C.CDLL) -> None:
    """Argument types of the tfx_rope functions (called once, by the package's loader)."""
    vp, i, l64 = C.c_void_p, C.c_int, C.c_int64
    L.tfx_rope_table.argtypes = [vp, i, vp]
    L.tfx_rope_apply.argtypes = [C.POINTER(RopeStruct), i, i, vp, l64, i, vp, l64, vp, l64, i, vp, l64, vp, i, i, vp]
    for n in ABI_SYMBOLS:
        getattr(L, n).restype = C.c_int


def rope_frequencies(rotary: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original: int = 4096, slow: float = 1.0, fast: float = 32.0) -> tuple:
    """(radians a position of each of the rotary/2 pairs, factor of the rotated values).

    Pair i has f_i = base^(-2i/rotary). scaling for contexts `factor` times as long as the
    `original` positions: "linear" divides every f_i by factor; "ntk" takes base *
    factor^(rotary/(rotary-2)); "yarn" keeps the pairs that turn more than `fast` times over the
    original positions, divides those that turn less than `slow` times, goes linearly from one
    to the other over the pairs between, and multiplies by 0.1 ln(factor) + 1.
    """
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling {scaling!r}: linear, ntk or yarn")
    if rotary < 4 or rotary % 2 or not base > 1 or not factor > 0 or not 0 < slow < fast or original < 1:
        raise ValueError("rotary is even and at least 4, base above 1, factor and original positive, 0 < slow < fast")
    gain = 1.0
    if scaling == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    f = [base ** (-2 * i / rotary) for i in range(rotary // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "yarn":
        def pair(turns):
            return rotary * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
        low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rotary - 1)
        part = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(rotary // 2)]
        f = [x * (1 - p) + x / factor * p for x, p in zip(f, part)]
        gain = 0.1 * math.log(factor) + 1
    return f, gain


class Rope:
    """Rotary positions of heads of `dim` values: the C descriptor and its table on a device.

    The first `rotary` values of a head (all by default; a multiple of 16) are rotated: value i
    with value i + rotary/2, or (interleaved) neighbours. Frequencies are rope_frequencies', or
    freqs (radians a position of each pair) and gain.
    """

    def __init__(self, dim: int, rotary: int | None = None, base: float = 10000.0, interleaved: bool = False,
                 scaling: str | None = None, factor: float = 1.0, original: int = 4096, slow: float = 1.0,
                 fast: float = 32.0, freqs=None, gain: float | None = None, device=None):
        if _at.torch is None:
            _at._load()
        torch = _at.torch
        rotary = dim if rotary is None else rotary
        _at._int32s(dim=dim, rotary=rotary)
        if rotary < 16 or rotary % 16 or rotary > dim or dim % 8:
            raise ValueError(f"rotary={rotary} of dim={dim}: rotary is a multiple of 16 and at most dim, dim one of 8")
        if freqs is None:
            freqs, own = rope_frequencies(rotary, base, scaling, factor, original, slow, fast)
            gain = own if gain is None else gain
        elif scaling is not None:
            raise ValueError("freqs are taken as they are: no scaling beside them")
        freqs = [float(f) for f in freqs]
        gain = 1.0 if gain is None else float(gain)
        if len(freqs) != rotary // 2:
            raise ValueError(f"{len(freqs)} frequencies, {rotary // 2} are wanted")
        n = len(freqs)
        table = (C.c_uint64 * n)()
        _at._check(_at._lib().tfx_rope_table((C.c_double * n)(*freqs), n, table))
        host = torch.tensor([x - (1 << 64) if x >> 63 else x for x in table], dtype=torch.int64)
        self.table = host.to("cuda" if device is None else device)
        self.dim, self.rotary, self.interleaved, self.gain, self.freqs = dim, rotary, bool(interleaved), gain, freqs
        self.device = self.table.get_device()
        if self.device < 0:
            raise ValueError("a CUDA device is wanted")
        self.s = RopeStruct(self.table.data_ptr(), rotary, int(interleaved), gain)
        self.ref = C.byref(self.s)


def rope(r: Rope, q, k, positions, out=None, inverse: bool = False, stream=None):
    """q (rows, heads, dim) and k (rows, kv_heads, dim; or None) with row t rotated to
    positions[t] (tfx_rope_apply; an int32 vector on the device). out: the tensors to write
    to, (q, k) themselves for a rotation in place, else none that overlaps an input; made here by default. inverse: by the
    negative angles. Returns (q, k)."""
    torch = _at.torch
    shape, dev, dtype, dim = q.shape, q.get_device(), q.dtype, r.dim
    if len(shape) != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k are (rows, heads, dim)")
    heads, kv = shape[1], 0 if k is None else k.shape[1]
    act = _at._act(dtype)
    rows, ldq, pq = _at._rows("q", q, heads, dim, dtype, dev)
    if dev != r.device:
        raise ValueError(f"q is on {q.device}, the table on CUDA device {r.device}")
    nk, ldk, pk = (rows, 0, None) if k is None else _at._rows("k", k, kv, dim, dtype, dev)
    n, pp = _at._ints("positions", positions, dev)
    if nk != rows or n != rows:
        raise ValueError(f"{rows} rows of q, {nk} of k, {n} positions")
    if heads >= _at._TOP or kv >= _at._TOP:
        _at._int32s(heads=heads, kv_heads=kv)
    on = _at._stream(stream, dev)
    if out is None:
        if stream is None:
            out = (torch.empty(shape, dtype=dtype, device=q.device),
                   None if k is None else torch.empty(k.shape, dtype=dtype, device=q.device))
        else:
            out = (_at._made_on(stream, dev, shape, dtype), None if k is None else _at._made_on(stream, dev, k.shape, dtype))
    qo, ko = out
    if (ko is None) != (k is None):
        raise ValueError("out holds a tensor for each of q and k")
    no, ldqo, pqo = _at._rows("out", qo, heads, dim, dtype, dev)
    mo, ldko, pko = (rows, 0, None) if ko is None else _at._rows("out", ko, kv, dim, dtype, dev)
    if no != rows or mo != rows:
        raise ValueError(f"out has {no} and {mo} rows, {rows} are wanted")
    rc = _at._lib().tfx_rope_apply(r.ref, act, dim, pq, ldq, heads, pqo, ldqo, pk, ldk, kv, pko, ldko, pp, rows, int(inverse), on)
    if rc:
        _at._check(rc)
    return qo, ko
