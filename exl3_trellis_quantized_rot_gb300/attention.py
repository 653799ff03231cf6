"""Python binding of the tfx_attn C ABI: attention and its paged K/V cache.

Argument marshalling and shape checks only, as in the package's linear layer:
every step runs in the kernels of ``libtfx_exl3.so``. Names follow the C ABI:
``attn_prompt``, ``attn_decode``, ``cache_reserve``, ``cache_release``,
``cache_extend``, ``cache_append``, ``cache_fork``, ``cache_free``,
``cache_compact``, ``cache_copy``.
"""
from __future__ import annotations

import ctypes as C

CACHE_FULL, CACHE_BAD, CACHE_TABLE_FULL = 1, 2, 4
MAX_BATCH = 4096

ABI_SYMBOLS = ("tfx_attn_prompt", "tfx_attn_decode", "tfx_attn_debug_error", "tfx_cache_book_ints", "tfx_cache_reserve",
               "tfx_cache_release", "tfx_cache_extend", "tfx_cache_append", "tfx_cache_fork", "tfx_cache_free",
               "tfx_cache_compact", "tfx_cache_copy")


class HeadsStruct(C.Structure):
    _fields_ = [("heads_q", C.c_int), ("heads_kv", C.c_int), ("dim", C.c_int), ("act", C.c_int), ("scale", C.c_float)]


class CacheStruct(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("book", C.c_void_p), ("layers", C.c_int), ("pages", C.c_int),
                ("page_size", C.c_int), ("heads_kv", C.c_int), ("dim", C.c_int), ("act", C.c_int), ("slots", C.c_int),
                ("width", C.c_int), ("priv", C.c_void_p)]


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
    L.tfx_cache_fork.argtypes = [K, vp, vp, i, vp]
    L.tfx_cache_free.argtypes = [K, vp, i, vp]
    L.tfx_cache_compact.argtypes = [K, vp]
    L.tfx_cache_copy.argtypes = [K, vp, vp, i, vp]
    for n in ABI_SYMBOLS:
        getattr(L, n).restype = C.c_int
    L.tfx_cache_book_ints.restype = l64


def _base():
    import exl3_trellis_quantized_rot_gb300 as tfx
    return tfx


def _act(dtype) -> int:
    import torch
    tfx = _base()
    if dtype == torch.float16:
        return tfx.F16
    if dtype == torch.bfloat16:
        return tfx.BF16
    raise ValueError(f"dtype {dtype}: float16 or bfloat16")


def _rows(name: str, t, heads: int, dim: int, like) -> None:
    """t is (rows, heads, dim) with whole rows (heads and values contiguous), on one device and in one type."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} of shape {tuple(t.shape)}: (rows, {heads}, {dim}) is wanted")
    if t.dtype != like.dtype or t.device != like.device or not t.is_cuda:
        raise ValueError(f"{name} is {t.dtype} on {t.device}, not {like.dtype} on {like.device} (a CUDA device)")
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim):
        raise ValueError(f"{name}: the heads of a row must lie next to each other")


def _pitch(t) -> int:
    # a single row's pitch is not used, and torch may give it any stride
    return t.stride(0) if t.shape[0] > 1 else max(8, t.shape[1] * t.shape[2])


def _ints(name: str, t, device) -> int:
    import torch
    if t.dtype != torch.int32 or t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1) or t.device != device:
        raise ValueError(f"{name}: a contiguous int32 vector on {device} is wanted")
    return t.data_ptr()


def attn_prompt(q, k, v, offsets, scale: float | None = None, out=None, stream=None):
    """Causal attention over packed prompts (tfx_attn_prompt). q: (T, heads, dim),
    k and v: (T, kv_heads, dim), rows any multiple of 8 values apart; offsets:
    int32 tensor on the CPU, sequence i is rows offsets[i]:offsets[i+1].
    scale: 1/sqrt(dim) by default. Returns out (rows outside the sequences of
    an out that is made here are zero)."""
    import torch
    tfx = _base()
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v are (rows, heads, dim)")
    T, hq, dim = q.shape
    hkv = k.shape[1]
    _rows("q", q, hq, dim, q)
    _rows("k", k, hkv, dim, q)
    _rows("v", v, hkv, dim, q)
    po = _ints("offsets", offsets, torch.device("cpu"))
    n = offsets.numel() - 1
    if n < 0:
        raise ValueError("offsets holds at least one value")
    first, last = int(offsets[0]), int(offsets[-1])
    if last > min(T, k.shape[0], v.shape[0]):
        raise ValueError(f"offsets end at {last}, past the rows of q, k or v")
    if out is None:
        out = torch.empty((T, hq, dim), dtype=q.dtype, device=q.device)
        if first > 0 or last < T:
            out.zero_()
    else:
        _rows("out", out, hq, dim, q)
        if out.shape[0] < last:
            raise ValueError(f"out has {out.shape[0]} rows, offsets end at {last}")
    h = HeadsStruct(hq, hkv, dim, _act(q.dtype), dim ** -0.5 if scale is None else scale)
    tfx._check(tfx.lib().tfx_attn_prompt(C.byref(h), q.data_ptr(), _pitch(q), k.data_ptr(), _pitch(k), v.data_ptr(),
                                         _pitch(v), po, n, out.data_ptr(), _pitch(out), tfx._stream(stream)))
    return out


class Cache:
    """A paged K/V cache: the C descriptor plus references keeping its tensors alive.

    k, v: (layers, pages, page_size, kv_heads, dim), contiguous; slots: sequences
    it can hold; width: pages that one sequence can have; book: int32 vector
    (made empty here by default), see ``lens``, ``refs`` and ``tables``.
    """

    def __init__(self, k, v, slots: int, width: int, book=None):
        import torch
        if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v are (layers, pages, page_size, kv_heads, dim), of one shape, type and device")
        if not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("k and v must be contiguous")
        layers, pages, page_size, heads, dim = k.shape
        self.s = CacheStruct(k.data_ptr(), v.data_ptr(), None, layers, pages, page_size, heads, dim, _act(k.dtype), slots,
                             width, None)
        ints = 4 + slots + pages + slots * width
        if book is None:
            book = torch.zeros(ints, dtype=torch.int32, device=k.device)
            book[4 + slots + pages:] = -1
        elif book.numel() != ints:
            raise ValueError(f"book of {book.numel()} values, {ints} are wanted")
        self.s.book = _ints("book", book, k.device)
        self.k, self.v, self.book = k, v, book

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

    def ref(self):
        return C.byref(self.s)

    def __del__(self):
        try:
            tfx = _base()
            if self.s.priv and tfx._lib is not None:
                tfx._lib.tfx_cache_release(C.byref(self.s))
        except Exception:
            pass


def cache_reserve(c: Cache, max_batch: int, heads: int, stream=None) -> None:
    """Scratch for attn_decode over up to max_batch sequences of `heads` query heads, and for the page calls."""
    tfx = _base()
    tfx._check(tfx.lib().tfx_cache_reserve(c.ref(), max_batch, heads, tfx._stream(stream)))


def cache_release(c: Cache) -> None:
    tfx = _base()
    tfx._check(tfx.lib().tfx_cache_release(c.ref()))


def cache_extend(c: Cache, seqs, offsets, stream=None) -> None:
    """Room for offsets[i+1] - offsets[i] new tokens of sequence seqs[i] (int32 vectors on the cache's device)."""
    tfx = _base()
    n = seqs.numel()
    if offsets.numel() != n + 1:
        raise ValueError(f"{offsets.numel()} offsets for {n} sequences")
    tfx._check(tfx.lib().tfx_cache_extend(c.ref(), _ints("seqs", seqs, c.k.device), _ints("offsets", offsets, c.k.device), n,
                                          tfx._stream(stream)))


def cache_append(c: Cache, layer: int, k, v, seqs=None, offsets=None, stream=None) -> None:
    """K and V (rows, kv_heads, dim) of one layer's new tokens, into the room that
    the last cache_extend made. seqs and offsets are that call's and may be left
    out: where each row goes was settled there."""
    tfx = _base()
    _rows("k", k, c.s.heads_kv, c.s.dim, c.k)
    _rows("v", v, c.s.heads_kv, c.s.dim, c.k)
    if k.shape[0] != v.shape[0]:
        raise ValueError(f"{k.shape[0]} rows of k, {v.shape[0]} of v")
    if offsets is not None and seqs is not None and offsets.numel() != seqs.numel() + 1:
        raise ValueError(f"{offsets.numel()} offsets for {seqs.numel()} sequences")
    tfx._check(tfx.lib().tfx_cache_append(c.ref(), layer, k.data_ptr(), _pitch(k), v.data_ptr(), _pitch(v), k.shape[0],
                                          tfx._stream(stream)))


def _pair(name: str, c: Cache, src, dst):
    if src.numel() != dst.numel():
        raise ValueError(f"{name}: {src.numel()} sources, {dst.numel()} targets")
    return _ints("src", src, c.k.device), _ints("dst", dst, c.k.device), src.numel()


def cache_fork(c: Cache, src, dst, stream=None) -> None:
    """Slot dst[i] becomes a copy of sequence src[i]: full pages shared, a partly filled last one copied."""
    tfx = _base()
    tfx._check(tfx.lib().tfx_cache_fork(c.ref(), *_pair("fork", c, src, dst), tfx._stream(stream)))


def cache_free(c: Cache, seqs, stream=None) -> None:
    """The sequences give their pages back."""
    tfx = _base()
    tfx._check(tfx.lib().tfx_cache_free(c.ref(), _ints("seqs", seqs, c.k.device), seqs.numel(), tfx._stream(stream)))


def cache_compact(c: Cache, stream=None) -> None:
    """Moves the used pages to the front of the pool; book[1] is the number moved."""
    tfx = _base()
    tfx._check(tfx.lib().tfx_cache_compact(c.ref(), tfx._stream(stream)))


def cache_copy(c: Cache, src, dst, stream=None) -> None:
    """Contents of page src[i] to page dst[i], all layers."""
    tfx = _base()
    tfx._check(tfx.lib().tfx_cache_copy(c.ref(), *_pair("copy", c, src, dst), tfx._stream(stream)))


def attn_decode(c: Cache, layer: int, q, seqs, shared: int = 0, scale: float | None = None, out=None, stream=None):
    """Attention of one new token of each sequence seqs[i] over the cache's tokens
    (tfx_attn_decode). q: (batch, heads, dim); the first `shared` tokens, the same
    in all of them, are read once. Returns out."""
    import torch
    tfx = _base()
    if q.dim() != 3:
        raise ValueError("q is (batch, heads, dim)")
    b, hq, dim = q.shape
    _rows("q", q, hq, c.s.dim, c.k)
    ps = _ints("seqs", seqs, c.k.device)
    if seqs.numel() != b:
        raise ValueError(f"{seqs.numel()} sequences for {b} rows of q")
    if out is None:
        out = torch.empty((b, hq, dim), dtype=q.dtype, device=q.device)
    else:
        _rows("out", out, hq, dim, q)
        if out.shape[0] != b:
            raise ValueError(f"out has {out.shape[0]} rows, q {b}")
    h = HeadsStruct(hq, c.s.heads_kv, dim, c.s.act, dim ** -0.5 if scale is None else scale)
    tfx._check(tfx.lib().tfx_attn_decode(c.ref(), layer, C.byref(h), q.data_ptr(), _pitch(q), ps, b, shared, out.data_ptr(),
                                         _pitch(out), tfx._stream(stream)))
    return out


def attn_error() -> int:
    """The attention kernels' device error word (0, or 1: a bounded wait gave up); reading clears it."""
    tfx = _base()
    e = C.c_int()
    tfx._check(tfx.lib().tfx_attn_debug_error(C.byref(e)))
    return e.value
