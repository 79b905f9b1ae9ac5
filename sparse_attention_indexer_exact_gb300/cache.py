"""The 4-bit paged cache and the attention that reads it at the selected entries.

Bindings of ``include/gvr_cache.h``, in the manner of the package's top-K calls: tensors are
checked and turned into addresses here, everything else happens in one kernel per call (two for
attention over whole caches of many entries) on the current stream of the tensors' device, or on the
one given as ``stream=`` to any of the calls.  They are for serving: no gradient passes through them.
A decode step, in call order::

    slots, counts = cache_tables(cached_lens, kv_lens, free_pages, block_table, new, page_size, cr)
    cache_append(k, v, cache, slots)                       # cache = cache_alloc(pages, page_size, heads, dim)
    idx, _ = topk_decode(logits, kv_lens, next_n, cr, K)
    out, _ = attend_decode(q, cache, block_table, kv_lens, next_n, cr, idx)

The cache is a uint8 tensor [pages, page_size, kv_heads, row]; ``include/gvr_cache.h`` has the
layout of a row, the quantiser and what every call does at its borders.
"""
from __future__ import annotations

import ctypes
import math
import operator
import warnings

__all__ = ["cache_alloc", "cache_row_bytes", "cache_tables", "cache_append", "cache_read", "attend_decode",
           "attend_prefill", "MAX_CACHE_REQUESTS", "HEAD_DIMS"]

HEAD_DIMS = (64, 128, 256)
MAX_CACHE_REQUESTS = 8192
_ROW_BYTES = {64: 80, 128: 144, 256: 288}
_HEAD_DIM = {row: dim for dim, row in _ROW_BYTES.items()}

EXPORTED_SYMBOLS = ("cache_row_bytes", "cache_tables", "cache_append", "cache_read", "attend_decode", "attend_prefill",
                    "gvr_cache_status_string")


class _Cache(ctypes.Structure):
    """Mirror of ``gvr_cache``."""
    _fields_ = [("data", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


def _declare(lib):
    i64, i32, p, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
    cache = ctypes.POINTER(_Cache)
    lib.cache_row_bytes.argtypes = [i32, ctypes.POINTER(i32)]
    lib.cache_tables.argtypes = [p, p, i64, i32, i32, p, i64, p, i64, i64, p, i64, p, p]
    lib.cache_append.argtypes = [cache, p, i64, i64, p, i64, i64, i32, p, i64, p]
    lib.cache_read.argtypes = [cache, p, i64, i32, p, p, p]
    sz = ctypes.c_size_t
    lib.attend_decode.argtypes = [cache, p, i64, i64, i32, i64, i32, p, i64, i64, p, i32, i32, p, i64, f32, p, p, p, sz, p]
    lib.attend_prefill.argtypes = [cache, p, i64, i64, i32, i64, i32, p, i64, i64, i64, p, p, p, p, i64, f32, p, p, p, sz, p]
    for name in EXPORTED_SYMBOLS[:-1]:
        getattr(lib, name).restype = ctypes.c_int
    lib.gvr_cache_status_string.argtypes = [ctypes.c_int]
    lib.gvr_cache_status_string.restype = ctypes.c_char_p


_WORKSPACE = 1 << 25  # GVR_ATTEND_WORKSPACE
# Selections over this many entries a row get a workspace, as whole caches do.  topk_decode and topk_prefill select up to
# 2048; longer ones come from elsewhere.  64 rows of 3000 entries, 64 heads over 8 of 128: 55 us with it, 61 without; one row of
# 3000 10.9 and 14.9.  Of 2048: 128 rows 70 and 76, but 37 rows under one KV head 19.8 and 18.3, 700 prefill rows 159 and 142.
_LONG = 2048

_lib = None


def _library():
    global _lib
    if _lib is None:
        from . import load_library
        _lib = load_library()
    return _lib


def _check(lib, status: int):
    if status != 0:
        from . import GvrError
        raise GvrError(status, lib.gvr_cache_status_string(status).decode())


def _launch(device: int, call, *args):
    """``call(*args, stream)`` on the current stream of the tensors' device, with that device current."""
    import torch
    stream = torch._C._cuda_getCurrentRawStream(device)
    if device == torch._C._cuda_getDevice():
        status = call(*args, stream)
    else:
        with torch.cuda.device(device):
            status = call(*args, stream)
    if status != 0:
        _check(_library(), status)


def _current(stream, tensor):
    """Context in which ``stream`` (a torch stream or a handle) is the current one: what a call
    allocates then belongs to the stream that uses it.  A handle does not tell its device: one of another
    device is refused by the launch."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        # handle 0 is the default stream; to ExternalStream it would mean a new one
        stream = torch.cuda.ExternalStream(stream, tensor.device) if int(stream) else torch.cuda.default_stream(tensor.device)
    if stream.device != tensor.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {tensor.device}")
    return torch.cuda.stream(stream)


# The short way (_native.cpp): the same calls with the tensors read natively.  Its functions return
# None wherever anything is out of the ordinary, and the call then goes step by step through the
# checks below, which say what is wrong.  Where it was not built every call does.
_native = None


class _NoShortWay:
    @staticmethod
    def _nothing(*args):
        return None

    cache_tables = cache_append = cache_read = attend_decode = attend_prefill = _nothing
    attend_shared = attend_weights = cache_evict = _nothing  # longcache.py


def _short():
    global _native
    if _native is None:
        _library()
        try:
            import torch  # noqa: F401 - its libraries have to be there first
            from . import _build
            from . import _native as native
            built_for = getattr(native, "BUILT_FOR", "an unknown torch")
            if built_for != _build.native_target():
                raise ImportError(f"built for {built_for}, this is {_build.native_target()}")
        except ImportError as e:
            warnings.warn(f"_native.so is missing or does not fit this torch ({e}): the cache calls take 15 us more of host "
                          "time; build it with `python -m sparse_attention_indexer_exact_gb300._build`", RuntimeWarning)
            native = _NoShortWay
        _native = native
    return _native


def _int32_value(value, name) -> int:
    """An integer that the library takes in 32 bits: ctypes would drop the bits above them."""
    value = operator.index(value)
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, {value} does not")
    return value


# The checks of one tensor: its device's number, or an error that names it.
def _device(t, name) -> int:
    import torch
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _on(t, device: int, name):
    if _device(t, name) != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not on cuda:{device}: all tensors must share one device")


def _int32(t, device: int, name, least=0) -> int:
    """Address of a contiguous 1-D int32 tensor of at least ``least`` entries."""
    import torch
    _on(t, device, name)
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    shape = t.shape
    if len(shape) != 1 or shape[0] < least or (shape[0] > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be 1-D contiguous with at least {least} entries")
    return t.data_ptr()


def _dtype(t, name) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float16:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float16")


def _heads_3d(t, name, dim):
    """(row stride, head stride) of [rows, heads, dim] with unit inner stride."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"{name} must be [rows, heads, {dim}]")
    if t.numel() == 0:
        return 0, 0
    row, head, inner = t.stride()
    if inner != 1:
        raise ValueError(f"{name} must have unit inner stride")
    # a dimension of one element is never stepped over
    return (row if shape[0] > 1 else 0), (head if shape[1] > 1 else 0)


def _table_2d(t, device: int, requests):
    """(address, stride, width) of an int32 block table [>= requests, width]."""
    import torch
    _on(t, device, "block_table")
    if t.dtype != torch.int32:
        raise TypeError("block_table must be int32")
    shape = t.shape
    if len(shape) != 2 or shape[0] < requests:
        raise ValueError(f"block_table must be [>= {requests}, pages] with unit inner stride")
    width = shape[1]
    row, inner = t.stride()
    if shape[0] > 0 and width > 1 and inner != 1:
        raise ValueError(f"block_table must be [>= {requests}, pages] with unit inner stride")
    return t.data_ptr(), (row if shape[0] > 1 else width), width


def _cache_struct(cache, k_scale, v_scale):
    import torch
    _device(cache, "cache")
    if cache.dtype != torch.uint8:
        raise TypeError("cache must be uint8")
    shape = cache.shape
    dim = _HEAD_DIM.get(shape[3]) if len(shape) == 4 else None
    if dim is None:
        raise ValueError("cache must be [pages, page_size, kv_heads, row] with row 80, 144 or 288 (cache_alloc)")
    pages, size, heads, row = shape
    page, entry, head, inner = cache.stride()
    if pages and (inner != 1 or (heads > 1 and head != row) or (size > 1 and entry != heads * row)):
        raise ValueError("the rows of a page of the cache must be packed; only its pages may lie apart")
    return _Cache(cache.data_ptr(), pages, page if pages > 1 else size * heads * row, size, heads, dim, 0, k_scale, v_scale)


def cache_row_bytes(head_dim: int) -> int:
    """Bytes of one entry of one KV head: K and V codes and scales of ``head_dim`` values."""
    lib = _library()
    out = ctypes.c_int32(0)
    _check(lib, lib.cache_row_bytes(_int32_value(head_dim, "head_dim"), ctypes.byref(out)))
    return out.value


def cache_alloc(num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, device="cuda"):
    """An empty cache: uint8 zeros [num_pages, page_size, num_kv_heads, row] (every value reads as 0)."""
    import torch
    return torch.zeros((num_pages, page_size, num_kv_heads, cache_row_bytes(head_dim)), dtype=torch.uint8, device=device)


def cache_tables(cached_lens, kv_lens, free_pages, block_table, max_new: int, page_size: int, compress_ratio: int = 1,
                 slots=None, counts=None, *, stream=None):
    """Give each request the pages that its new entries need, and map those entries to slots.

    ``cached_lens`` and ``kv_lens`` (int32 [requests]) are each request's uncompressed length before
    and after the step; ``block_table`` (int32 [requests, width]) is extended in place with pages
    from ``free_pages`` (int32).  Returns ``slots`` (int32 [max_new], the new entries' slots in
    order, -1 behind them and where no page was left) and ``counts`` (int32 [3]: new entries, pages
    taken, pages missing).
    """
    if stream is not None:
        with _current(stream, kv_lens):
            return cache_tables(cached_lens, kv_lens, free_pages, block_table, max_new, page_size, compress_ratio, slots, counts)
    done = (_native or _short()).cache_tables(cached_lens, kv_lens, free_pages, block_table, max_new, page_size,
                                              compress_ratio, slots, counts)
    if done is not None:
        return done
    import torch
    page_size, compress_ratio = _int32_value(page_size, "page_size"), _int32_value(compress_ratio, "compress_ratio")
    device = _device(kv_lens, "kv_lens")
    requests = kv_lens.shape[0] if kv_lens.dim() == 1 else 0
    lens = _int32(kv_lens, device, "kv_lens")
    cached = _int32(cached_lens, device, "cached_lens", requests)
    free = _int32(free_pages, device, "free_pages")
    table, table_stride, width = _table_2d(block_table, device, requests)
    if slots is None:
        slots = torch.empty(max_new, dtype=torch.int32, device=kv_lens.device)
        to = slots.data_ptr()
    else:
        to = _int32(slots, device, "slots", max_new)
    if counts is None:
        counts = torch.empty(3, dtype=torch.int32, device=kv_lens.device)
        sums = counts.data_ptr()
    else:
        sums = _int32(counts, device, "counts", 3)
    _launch(device, _library().cache_tables, cached, lens, requests, compress_ratio, page_size, free,
            free_pages.shape[0], table, table_stride, width, to, max_new, sums)
    return slots, counts


def cache_append(k, v, cache, slots, *, k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Quantise ``k`` and ``v`` [tokens, kv_heads, head_dim] (bfloat16 or float16, strides in multiples
    of 8) into ``cache`` at ``slots`` (int32 [tokens]; -1 skips the token)."""
    if stream is not None:
        with _current(stream, cache):
            return cache_append(k, v, cache, slots, k_scale=k_scale, v_scale=v_scale)
    if (_native or _short()).cache_append(k, v, cache, slots, k_scale, v_scale):
        return
    c = _cache_struct(cache, k_scale, v_scale)
    device = cache.get_device()
    _on(k, device, "k")
    _on(v, device, "v")
    kind = _dtype(k, "k")
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must have one shape and dtype")
    k_token, k_head = _heads_3d(k, "k", c.head_dim)
    v_token, v_head = _heads_3d(v, "v", c.head_dim)
    tokens, heads, _ = k.shape
    if heads != c.num_kv_heads:
        raise ValueError(f"k has {heads} heads, the cache {c.num_kv_heads}")
    at = _int32(slots, device, "slots", tokens)
    _launch(device, _library().cache_append, c, k.data_ptr(), k_token, k_head, v.data_ptr(), v_token, v_head, kind,
            at, tokens)


def cache_read(cache, slots, head_dim: int, dtype=None, *, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """The values held at ``slots`` (int32 [n]): K and V, each [n, kv_heads, head_dim] of ``dtype``
    (bfloat16 by default, or float16); zeros for a slot that names no entry."""
    import torch
    if stream is not None:
        with _current(stream, cache):
            return cache_read(cache, slots, head_dim, dtype, k_scale=k_scale, v_scale=v_scale)
    kind = 0 if dtype is None or dtype == torch.bfloat16 else 1 if dtype == torch.float16 else -1
    done = (_native or _short()).cache_read(cache, slots, head_dim, kind, k_scale, v_scale)
    if done is not None:
        return done
    c = _cache_struct(cache, k_scale, v_scale)
    device = cache.get_device()
    if c.head_dim != head_dim:
        raise ValueError(f"the cache holds heads of {c.head_dim}, not {head_dim}")
    at = _int32(slots, device, "slots")
    n = slots.shape[0]
    kv = torch.empty((2, n, c.num_kv_heads, head_dim), dtype=dtype or torch.bfloat16, device=cache.device)
    k, v = kv.unbind(0)
    _launch(device, _library().cache_read, c, at, n, _dtype(kv, "dtype"), k.data_ptr(), v.data_ptr())
    return k, v


def _attend(q, cache, k_scale, v_scale, scale, out, lse, want_lse):
    """What both attention calls check: the arguments up to the block table, and the outputs."""
    import torch
    c = _cache_struct(cache, k_scale, v_scale)
    device = cache.get_device()
    _on(q, device, "q")
    kind = _dtype(q, "q")
    row, head = _heads_3d(q, "q", c.head_dim)
    rows, heads, dim = q.shape
    if heads == 0 or heads % c.num_kv_heads:
        raise ValueError(f"q has {heads} heads, no multiple of the cache's {c.num_kv_heads}")
    if out is None:
        out = torch.empty((rows, heads, dim), dtype=q.dtype, device=q.device)
    else:
        _on(out, device, "out")
        if out.dtype != q.dtype or out.shape != q.shape or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous {q.dtype} tensor of shape {tuple(q.shape)}")
    if lse is not None:
        _on(lse, device, "lse")
        if lse.dtype != torch.float32 or lse.shape != (rows, heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 tensor of shape ({rows}, {heads})")
    elif want_lse:
        lse = torch.empty((rows, heads), dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(dim)
    return device, (c, q.data_ptr(), row, head, kind, rows, heads), scale, out, lse


def _workspace(device):
    """Scratch of one call (32 MB): from torch's allocator, so each call on each stream has its own, and
    a captured graph keeps its own."""
    import torch
    return torch.empty(_WORKSPACE, dtype=torch.uint8, device=device)


def _indices_2d(t, device: int, rows):
    import torch
    _on(t, device, "indices")
    if t.dtype != torch.int32:
        raise TypeError("indices must be int32")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < 1 or not t.is_contiguous():
        raise ValueError(f"indices must be contiguous [{rows}, >= 1]")
    return t.data_ptr(), shape[1]


def attend_decode(q, cache, block_table, kv_lens, next_n: int, compress_ratio: int, indices=None, *, scale=None,
                  k_scale: float = 1.0, v_scale: float = 1.0, out=None, lse=None, want_lse: bool = False, stream=None):
    """Attention of decode rows over the 4-bit cache; returns (out, lse or None).

    ``q`` is [rows, heads, head_dim] (bfloat16 or float16, strides in multiples of 8); row r belongs to
    request r // next_n (``next_n`` up to 4096) and sees its (kv_len - next_n + r % next_n + 1) // compress_ratio entries, found
    through ``block_table`` (int32 [requests, pages]): those that ``indices`` (int32 [rows, k], as
    ``topk_decode`` returns them) lists, or all where it is None.  ``scale`` defaults to
    1 / sqrt(head_dim).  ``lse`` (fp32 [rows, heads]) is the log of each row's sum of exponentials.
    """
    if stream is not None:
        with _current(stream, q):
            return attend_decode(q, cache, block_table, kv_lens, next_n, compress_ratio, indices, scale=scale, k_scale=k_scale,
                                 v_scale=v_scale, out=out, lse=lse, want_lse=want_lse)
    done = (_native or _short()).attend_decode(q, cache, k_scale, v_scale, scale, out, lse, want_lse, block_table, kv_lens,
                                               next_n, compress_ratio, indices)
    if done is not None:
        return done
    next_n, compress_ratio = _int32_value(next_n, "next_n"), _int32_value(compress_ratio, "compress_ratio")
    device, head, scale, out, lse = _attend(q, cache, k_scale, v_scale, scale, out, lse, want_lse)
    rows = head[5]
    requests = (rows + next_n - 1) // max(next_n, 1)
    table, table_stride, width = _table_2d(block_table, device, requests)
    lens = _int32(kv_lens, device, "kv_lens", requests)
    listed, k = (None, 0) if indices is None else _indices_2d(indices, device, rows)
    space = _workspace(q.device) if k == 0 or k > _LONG else None
    _launch(device, _library().attend_decode, *head, table, table_stride, width, lens, next_n, compress_ratio,
            listed, k, scale, out.data_ptr(), None if lse is None else lse.data_ptr(),
            None if space is None else space.data_ptr(), _WORKSPACE)
    return out, lse


def attend_prefill(q, cache, block_table, row_requests, row_starts, row_ends, indices, *, scale=None,
                   k_scale: float = 1.0, v_scale: float = 1.0, out=None, lse=None, want_lse: bool = False, stream=None):
    """Attention of prefill rows over their selection in the 4-bit cache; returns (out, lse or None).

    Row r belongs to request ``row_requests[r]`` (int32; outside the block table: no entries) and sees
    its first ``row_ends[r] - row_starts[r]`` entries, the window given to ``topk_prefill``, whose
    ``indices`` (int32 [rows, k]) it attends to.  The rest is as in :func:`attend_decode`.
    """
    if stream is not None:
        with _current(stream, q):
            return attend_prefill(q, cache, block_table, row_requests, row_starts, row_ends, indices, scale=scale,
                                  k_scale=k_scale, v_scale=v_scale, out=out, lse=lse, want_lse=want_lse)
    done = (_native or _short()).attend_prefill(q, cache, k_scale, v_scale, scale, out, lse, want_lse, block_table,
                                                row_requests, row_starts, row_ends, indices)
    if done is not None:
        return done
    device, head, scale, out, lse = _attend(q, cache, k_scale, v_scale, scale, out, lse, want_lse)
    rows = head[5]
    table, table_stride, width = _table_2d(block_table, device, 0)
    requests = _int32(row_requests, device, "row_requests", rows)
    starts = _int32(row_starts, device, "row_starts", rows)
    ends = _int32(row_ends, device, "row_ends", rows)
    listed, k = _indices_2d(indices, device, rows)
    space = _workspace(q.device) if k > _LONG else None
    _launch(device, _library().attend_prefill, *head, table, table_stride, width, block_table.shape[0], requests,
            starts, ends, listed, k, scale, out.data_ptr(), None if lse is None else lse.data_ptr(),
            None if space is None else space.data_ptr(), _WORKSPACE)
    return out, lse
