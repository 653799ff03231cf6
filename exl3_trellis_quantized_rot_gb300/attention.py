"""Python binding of the tfx_attn C ABI: attention and its paged K/V cache.

Argument marshalling and shape checks only, as in the package's linear layer:
every step runs in the kernels of ``libtfx_exl3.so``. Names follow the C ABI:
``attn_prompt``, ``attn_decode``, ``cache_reserve``, ``cache_release``,
``cache_extend``, ``cache_append``, ``cache_read``, ``cache_fork``, ``cache_free``,
``cache_compact``, ``cache_copy``.
"""
from __future__ import annotations

import ctypes as C
import functools
import sys

_pkg = sys.modules[__package__]  # being imported when this runs: its functions are looked up at each call

CACHE_FULL, CACHE_BAD, CACHE_TABLE_FULL = 1, 2, 4
STORE_ACT, STORE_I8, STORE_E4M3 = 0, 1, 2
CACHE_BLOCK = 16  # tokens of a head that share a scale in an 8-bit cache
MAX_BATCH = 4096
_TOP = 1 << 31

ABI_SYMBOLS = ("tfx_attn_prompt", "tfx_attn_decode", "tfx_attn_debug_error", "tfx_cache_book_ints", "tfx_cache_reserve",
               "tfx_cache_release", "tfx_cache_extend", "tfx_cache_append", "tfx_cache_append_listed", "tfx_cache_read",
               "tfx_cache_fork", "tfx_cache_free", "tfx_cache_compact", "tfx_cache_copy")


class HeadsStruct(C.Structure):
    _fields_ = [("heads_q", C.c_int), ("heads_kv", C.c_int), ("dim", C.c_int), ("act", C.c_int), ("scale", C.c_float)]


class CacheStruct(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("book", C.c_void_p), ("layers", C.c_int), ("pages", C.c_int),
                ("page_size", C.c_int), ("heads_kv", C.c_int), ("dim", C.c_int), ("act", C.c_int), ("slots", C.c_int),
                ("width", C.c_int), ("priv", C.c_void_p), ("store", C.c_int), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p)]


def declare(L: C.CDLL) -> None:
    """Argument types of the tfx_attn / tfx_cache functions (called once, by the package's loader)."""
    H, K, vp, i, l64 = C.POINTER(HeadsStruct), C.POINTER(CacheStruct), C.c_void_p, C.c_int, C.c_int64
    L.tfx_attn_prompt.argtypes = [H, vp, l64, vp, l64, vp, l64, vp, i, vp, l64, vp]
    L.tfx_attn_decode.argtypes = [K, i, H, vp, l64, vp, i, i, vp, l64, vp]
    L.tfx_attn_debug_error.argtypes = [C.POINTER(i)]
    L.tfx_cache_book_ints.argtypes = [K]
    L.tfx_cache_reserve.argtypes = [K, i, i, vp]
    L.tfx_cache_release.argtypes = [K]
    L.tfx_cache_extend.argtypes = [K, vp, vp, i, vp]
    L.tfx_cache_append.argtypes = [K, i, vp, l64, vp, l64, i, vp]
    L.tfx_cache_append_listed.argtypes = [K, i, vp, l64, vp, l64, i, vp, vp, i, vp]
    L.tfx_cache_read.argtypes = [K, i, vp, vp, vp, i, i, vp, l64, vp, l64, vp]
    L.tfx_cache_fork.argtypes = [K, vp, vp, i, vp]
    L.tfx_cache_free.argtypes = [K, vp, i, vp]
    L.tfx_cache_compact.argtypes = [K, vp]
    L.tfx_cache_copy.argtypes = [K, vp, vp, i, vp]
    for n in ABI_SYMBOLS:
        getattr(L, n).restype = C.c_int
    L.tfx_cache_book_ints.restype = l64


# Set by _load: the package imports without torch; what takes its tensors brings it in.
torch = _int32 = _raw_stream = _current_device = None
_act_of: dict = {}
_store_of: dict = {}


def _load() -> None:
    """Called where the first tensors arrive: by attn_prompt and by Cache, which every other call takes."""
    global torch, _int32, _raw_stream, _current_device
    import torch
    _act_of.update({torch.float16: 0, torch.bfloat16: 1})  # TFX_F16, TFX_BF16
    _store_of.update({torch.int8: STORE_I8, torch.float8_e4m3fn: STORE_E4M3})
    _int32 = torch.int32
    # absent without CUDA
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _current_device = getattr(torch._C, "_cuda_getDevice", None)


def _lib():
    return _pkg._lib or _pkg.lib()


@functools.lru_cache(maxsize=64)
def _heads(hq: int, hkv: int, dim: int, act: int, scale):
    """The C descriptor of a head layout (a model has a few); read-only once made, so
    scale is a float or None: a tensor would be told by its identity."""
    return C.byref(HeadsStruct(hq, hkv, dim, act, dim ** -0.5 if scale is None else scale))


def _check(rc: int) -> None:
    if rc:
        raise _pkg.TfxError(rc, _pkg.last_error())


def _stream(stream, device: int) -> int:
    """A stream's handle; by default torch's current one on the device, which must be
    the current device: that is where the library launches."""
    if _current_device() != device:
        raise ValueError(f"tensors on CUDA device {device}, the current one is {_current_device()}")
    return _raw_stream(device) if stream is None else stream if isinstance(stream, int) else stream.cuda_stream


def _int32s(**numbers) -> None:
    """Refuses numbers that a C int would take modulo 2^32."""
    for name, n in numbers.items():
        if not -_TOP <= n < _TOP:
            raise ValueError(f"{name}={n} does not fit 32 bits")


def _made_on(stream, device: int, shape: tuple, dtype, clear: bool = False):
    """A result for a call on a stream that the caller names: allocated, and cleared,
    in that stream's order, and known to the current one, where it will be read."""
    handle = _stream(stream, device)
    if isinstance(stream, torch.cuda.Stream):
        st = stream
    elif handle == 0:  # ExternalStream takes 0 for a new stream
        st = torch.cuda.default_stream(device)
    else:
        st = torch.cuda.ExternalStream(handle, device=device)
    with torch.cuda.stream(st):
        out = (torch.zeros if clear else torch.empty)(shape, dtype=dtype, device=f"cuda:{device}")
    out.record_stream(torch.cuda.current_stream(device))
    return out


def _act(dtype) -> int:
    act = _act_of.get(dtype)
    if act is None:
        raise ValueError(f"dtype {dtype}: float16 or bfloat16")
    return act


def _rows(name: str, t, heads: int, dim: int, dtype, device: int) -> tuple:
    """Checks that t is (rows, heads, dim) with whole rows (heads and values lie next
    to each other) of a type and on a CUDA device; (rows, pitch, address)."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} of shape {tuple(shape)}: (rows, {heads}, {dim}) is wanted")
    if t.dtype is not dtype or device < 0 or t.get_device() != device:
        raise ValueError(f"{name} is {t.dtype} on {t.device}: {dtype} on CUDA device {device} is wanted")
    row, head, value = t.stride()
    if value != 1 or (head != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a row must lie next to each other")
    # a single row's pitch is not used, and torch may give it any stride
    return shape[0], row if shape[0] > 1 else heads * dim, t.data_ptr()


def _ints(name: str, t, device: int) -> tuple:
    """(length, address) of a contiguous int32 vector; device -1 is the CPU."""
    if t.dtype is not _int32 or t.get_device() != device or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 vector on {'the CPU' if device < 0 else f'CUDA device {device}'} is wanted")
    n = t.numel()
    if n >= _TOP:  # the library counts in 32 bits
        raise ValueError(f"{name} of {n} values: fewer than 2^31 are wanted")
    return n, t.data_ptr()


def attn_prompt(q, k, v, offsets, scale: float | None = None, out=None, stream=None):
    """Causal attention over packed prompts (tfx_attn_prompt). q: (T, heads, dim),
    k and v: (T, kv_heads, dim), rows any multiple of 8 values apart; offsets:
    int32 tensor on the CPU, sequence i is rows offsets[i]:offsets[i+1].
    scale: 1/sqrt(dim) by default. Returns out (rows outside the sequences of
    an out that is made here are zero)."""
    if torch is None:
        _load()
    try:
        (T, hq, dim), (Tk, hkv, dk), (Tv, hv, dv) = q.shape, k.shape, v.shape
        (ldq, sq, eq), (ldk, sk, ek), (ldv, sv, ev) = q.stride(), k.stride(), v.stride()
    except ValueError:
        raise ValueError("q, k and v are (rows, heads, dim)") from None
    dtype, dev = q.dtype, q.get_device()
    # _rows' conditions all at once (short prompts wait for this code); what does not
    # meet them is looked at one by one: refused with the reason, or odd strides of a
    # dimension of one
    if (dim == dk == dv == sq == sk == sv and hv == hkv and eq == ek == ev == 1 and T > 1 and Tk > 1 and Tv > 1
            and k.dtype is dtype and v.dtype is dtype and k.get_device() == dev == v.get_device() and dev >= 0):
        pq, pk, pv = q.data_ptr(), k.data_ptr(), v.data_ptr()
    else:
        T, ldq, pq = _rows("q", q, hq, dim, dtype, dev)
        Tk, ldk, pk = _rows("k", k, hkv, dim, dtype, dev)
        Tv, ldv, pv = _rows("v", v, hkv, dim, dtype, dev)
    if scale is not None:
        scale = float(scale)
    n, po = _ints("offsets", offsets, -1)
    if n < 1:
        raise ValueError("offsets holds at least one value")
    first, last = C.c_int32.from_address(po).value, C.c_int32.from_address(po + 4 * (n - 1)).value
    if last > T or last > Tk or last > Tv:
        raise ValueError(f"offsets end at {last}, past the rows of q, k or v")
    if out is None:
        clear = first > 0 or last < T
        if stream is None:
            out = torch.empty((T, hq, dim), dtype=dtype, device=q.device)
            if clear:
                out.zero_()
        else:
            out = _made_on(stream, dev, (T, hq, dim), dtype, clear)
        ldo, pout = hq * dim, out.data_ptr()
    else:
        To, ldo, pout = _rows("out", out, hq, dim, dtype, dev)
        if To < last:
            raise ValueError(f"out has {To} rows, offsets end at {last}")
    rc = (_pkg._lib or _pkg.lib()).tfx_attn_prompt(
        _heads(hq, hkv, dim, _act(dtype), scale), pq, ldq, pk, ldk, pv, ldv, po, n - 1, pout, ldo,
        _stream(stream, dev))
    if rc:
        _check(rc)
    return out


class Cache:
    """A paged K/V cache: the C descriptor plus references keeping its tensors alive.

    k, v: (layers, pages, page_size, kv_heads, dim), contiguous; slots: sequences
    it can hold; width: pages that one sequence can have; book: int32 vector
    (made empty here by default), see ``lens``, ``refs`` and ``tables``.

    k and v of int8 or float8_e4m3fn are a cache of 8-bit codes: act is the type of
    the rows that calls take and give (float16 or bfloat16), k_scale and v_scale are
    float32 (layers, pages, page_size / 16, kv_heads), contiguous (made here by
    default): a power of two for each 16 tokens of a head.
    """

    def __init__(self, k, v, slots: int, width: int, book=None, k_scale=None, v_scale=None, act=None):
        if torch is None:
            _load()
        if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v are (layers, pages, page_size, kv_heads, dim), of one shape, type and device")
        if not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("k and v must be contiguous")
        layers, pages, page_size, heads, dim = k.shape
        store = _store_of.get(k.dtype, STORE_ACT)
        if store == STORE_ACT:
            if act not in (None, k.dtype) or k_scale is not None or v_scale is not None:
                raise ValueError(f"act and scales go with k and v of int8 or float8_e4m3fn, not {k.dtype}")
            act = k.dtype
        elif act is None:
            raise ValueError(f"k and v of {k.dtype}: act says the type of the rows")
        self.s = CacheStruct(k.data_ptr(), v.data_ptr(), None, layers, pages, page_size, heads, dim, _act(act), slots,
                             width, None, store, None, None)
        ints = 4 + slots + pages + slots * width
        if book is None:
            book = torch.zeros(ints, dtype=torch.int32, device=k.device)
            book[4 + slots + pages:] = -1
        elif book.numel() != ints:
            raise ValueError(f"book of {book.numel()} values, {ints} are wanted")
        self.device, self.dtype, self.heads_kv, self.dim, self.act = k.get_device(), act, heads, dim, self.s.act
        self.ref = C.byref(self.s)
        self.s.book = _ints("book", book, self.device)[1]
        if store != STORE_ACT:
            shape = (layers, pages, page_size // CACHE_BLOCK, heads)
            k_scale, v_scale = (torch.zeros(shape, dtype=torch.float32, device=k.device) if t is None else t
                                for t in (k_scale, v_scale))
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if tuple(t.shape) != shape or t.dtype != torch.float32 or t.get_device() != self.device or not t.is_contiguous():
                    raise ValueError(f"{name}: a contiguous float32 tensor of shape {shape} on the cache's device is wanted")
            self.s.k_scale, self.s.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
        self.k, self.v, self.book, self.k_scale, self.v_scale = k, v, book, k_scale, v_scale

    @property
    def lens(self):
        return self.book[4:4 + self.s.slots]

    @property
    def refs(self):
        return self.book[4 + self.s.slots:4 + self.s.slots + self.s.pages]

    @property
    def tables(self):
        return self.book[4 + self.s.slots + self.s.pages:].view(self.s.slots, self.s.width)

    def status(self) -> int:
        """The book's status bits (CACHE_FULL, CACHE_BAD, CACHE_TABLE_FULL); waits for the GPU."""
        return int(self.book[0])

    def __del__(self):
        try:
            if self.s.priv and _pkg._lib is not None:
                _pkg._lib.tfx_cache_release(C.byref(self.s))
        except Exception:
            pass


def cache_reserve(c: Cache, max_batch: int, heads: int, stream=None) -> None:
    """Scratch for attn_decode over up to max_batch sequences of `heads` query heads, and for the page calls."""
    _int32s(max_batch=max_batch, heads=heads)
    _check(_lib().tfx_cache_reserve(c.ref, max_batch, heads, _stream(stream, c.device)))


def cache_release(c: Cache) -> None:
    _check(_lib().tfx_cache_release(c.ref))


def cache_extend(c: Cache, seqs, offsets, stream=None) -> None:
    """Room for offsets[i+1] - offsets[i] new tokens of sequence seqs[i] (int32 vectors
    on the cache's device). Behind one that finds too few pages, all that need any are
    refused: put first what must not be."""
    n, ps = _ints("seqs", seqs, c.device)
    m, po = _ints("offsets", offsets, c.device)
    if m != n + 1:
        raise ValueError(f"{m} offsets for {n} sequences")
    _check(_lib().tfx_cache_extend(c.ref, ps, po, n, _stream(stream, c.device)))


def cache_append(c: Cache, layer: int, k, v, seqs=None, offsets=None, stream=None) -> None:
    """K and V (rows, kv_heads, dim) of one layer's new tokens, into the room that
    cache_extend made, quantised on the way into a cache of 8-bit codes. seqs and offsets
    (int32 vectors on the cache's device) are that call's, or some entries of it; left out,
    the last cache_extend's."""
    if not -_TOP <= layer < _TOP:
        _int32s(layer=layer)
    heads, dim, dtype, dev = c.heads_kv, c.dim, c.dtype, c.device
    try:
        (n, hk, dk), (m, hv, dv), (ldk, sk, ek), (ldv, sv, ev) = k.shape, v.shape, k.stride(), v.stride()
    except ValueError:
        raise ValueError(f"k and v are (rows, {heads}, {dim})") from None
    # as in attn_prompt: _rows' conditions all at once
    if (n == m and hk == hv == heads and dim == dk == dv == sk == sv and ek == ev == 1
            and k.dtype is dtype and v.dtype is dtype and k.get_device() == dev == v.get_device() and dev >= 0):
        if n <= 1:  # a single row's pitch is not used
            ldk = ldv = heads * dim
        pk, pv = k.data_ptr(), v.data_ptr()
    else:
        n, ldk, pk = _rows("k", k, heads, dim, dtype, dev)
        m, ldv, pv = _rows("v", v, heads, dim, dtype, dev)
        if n != m:
            raise ValueError(f"{n} rows of k, {m} of v")
    on = _stream(stream, dev)
    if seqs is None and offsets is None:
        rc = (_pkg._lib or _pkg.lib()).tfx_cache_append(c.ref, layer, pk, ldk, pv, ldv, n, on)
    elif seqs is None or offsets is None:
        raise ValueError("seqs and offsets go together")
    else:
        ns, ps = _ints("seqs", seqs, dev)
        no, po = _ints("offsets", offsets, dev)
        if no != ns + 1:
            raise ValueError(f"{no} offsets for {ns} sequences")
        rc = (_pkg._lib or _pkg.lib()).tfx_cache_append_listed(c.ref, layer, pk, ldk, pv, ldv, n, ps, po, ns, on)
    if rc:
        _check(rc)


def cache_read(c: Cache, layer: int, seqs, starts, offsets, rows: int, out=None, stream=None):
    """K and V (rows, kv_heads, dim) of one layer out of the cache, in its act type: rows
    offsets[i]:offsets[i+1] are tokens starts[i], starts[i] + 1, ... of sequence seqs[i]
    (int32 vectors on the cache's device). out: a pair to write to; rows outside the lists
    stay as they are there, and are zero where it is made here. Returns (k, v)."""
    _int32s(layer=layer, rows=rows)
    dev = c.device
    n, ps = _ints("seqs", seqs, dev)
    m, pb = _ints("starts", starts, dev)
    no, po = _ints("offsets", offsets, dev)
    if m != n or no != n + 1:
        raise ValueError(f"{m} starts and {no} offsets for {n} sequences")
    if rows < 0:
        raise ValueError(f"rows={rows}")
    on = _stream(stream, dev)
    if out is None:
        shape = rows, c.heads_kv, c.dim
        if stream is None:
            out = tuple(torch.zeros(shape, dtype=c.dtype, device=c.k.device) for _ in range(2))
        else:
            out = tuple(_made_on(stream, dev, shape, c.dtype, True) for _ in range(2))
    k, v = out
    nk, ldk, pk = _rows("k", k, c.heads_kv, c.dim, c.dtype, dev)
    nv, ldv, pv = _rows("v", v, c.heads_kv, c.dim, c.dtype, dev)
    if nk < rows or nv < rows:
        raise ValueError(f"out has {nk} and {nv} rows, {rows} are wanted")
    rc = (_pkg._lib or _pkg.lib()).tfx_cache_read(c.ref, layer, ps, pb, po, n, rows, pk, ldk, pv, ldv, on)
    if rc:
        _check(rc)
    return k, v


def _pair(c: Cache, src, dst) -> tuple:
    n, ps = _ints("src", src, c.device)
    m, pd = _ints("dst", dst, c.device)
    if n != m:
        raise ValueError(f"{n} sources, {m} targets")
    return ps, pd, n


def cache_fork(c: Cache, src, dst, stream=None) -> None:
    """Slot dst[i] becomes a copy of sequence src[i]: full pages shared, a partly filled last one copied."""
    _check(_lib().tfx_cache_fork(c.ref, *_pair(c, src, dst), _stream(stream, c.device)))


def cache_free(c: Cache, seqs, stream=None) -> None:
    """The sequences give their pages back."""
    n, ps = _ints("seqs", seqs, c.device)
    _check(_lib().tfx_cache_free(c.ref, ps, n, _stream(stream, c.device)))


def cache_compact(c: Cache, stream=None) -> None:
    """Moves the used pages to the front of the pool; book[1] is the number moved."""
    _check(_lib().tfx_cache_compact(c.ref, _stream(stream, c.device)))


def cache_copy(c: Cache, src, dst, stream=None) -> None:
    """Contents of page src[i] to page dst[i], all layers."""
    _check(_lib().tfx_cache_copy(c.ref, *_pair(c, src, dst), _stream(stream, c.device)))


def attn_decode(c: Cache, layer: int, q, seqs, shared: int = 0, scale: float | None = None, out=None, stream=None):
    """Attention of one new token of each sequence seqs[i] over the cache's tokens
    (tfx_attn_decode). q: (batch, heads, dim); the first `shared` tokens, the same
    in all of them, are read once where the batch has many rows. Returns out."""
    try:
        (b, hq, dq), (ldq, sq, eq) = q.shape, q.stride()
    except ValueError:
        raise ValueError("q is (batch, heads, dim)") from None
    if not (-_TOP <= layer < _TOP and -_TOP <= shared < _TOP):
        _int32s(layer=layer, shared=shared)
    dim, dtype, dev = c.dim, c.dtype, c.device
    # as in attn_prompt: _rows' conditions all at once
    if dim == dq == sq and eq == 1 and q.dtype is dtype and q.get_device() == dev and dev >= 0:
        if b <= 1:
            ldq = hq * dim
        pq = q.data_ptr()
    else:
        b, ldq, pq = _rows("q", q, hq, dim, dtype, dev)
    if scale is not None:
        scale = float(scale)
    n, ps = _ints("seqs", seqs, dev)
    if n != b:
        raise ValueError(f"{n} sequences for {b} rows of q")
    if out is None:
        shape = b, hq, dim
        out = torch.empty(shape, dtype=dtype, device=q.device) if stream is None else _made_on(stream, dev, shape, dtype)
        ldo, po = hq * dim, out.data_ptr()
    else:
        bo, ldo, po = _rows("out", out, hq, dim, dtype, dev)
        if bo != b:
            raise ValueError(f"out has {bo} rows, q {b}")
    rc = (_pkg._lib or _pkg.lib()).tfx_attn_decode(c.ref, layer, _heads(hq, c.heads_kv, dim, c.act, scale), pq, ldq, ps, b,
                                                   shared, po, ldo, _stream(stream, dev))
    if rc:
        _check(rc)
    return out


def attn_error() -> int:
    """The attention kernels' device error word (0, or 1: a bounded wait gave up); reading clears it."""
    e = C.c_int()
    _check(_lib().tfx_attn_debug_error(C.byref(e)))
    return e.value
