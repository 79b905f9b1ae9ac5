"""Caches that live long: attention of requests that share prefixes, what each entry draws, eviction.

Bindings of ``include/gvr_long.h``, in the manner of ``cache.py`` and over the same 4-bit cache.  They are
for serving: no gradient passes through them.  A layer that reads its whole cache, in call order::

    out, lse = attend_shared(q, cache, block_table, kv_lens, next_n, cr, group_starts, prefix_entries, want_lse=True)
    attend_weights(q, cache, block_table, kv_lens, next_n, cr, lse, weights)      # weights += what each entry drew

and once the caches have grown over their budget::

    kept, kv_lens, released, counts = cache_evict(weights, cache, block_table, kv_lens, free_pages, keep, recent, cr)
"""
from __future__ import annotations

import ctypes
import math

from . import cache as _c
from .cache import _attend, _Cache, _cache_struct, _current, _device, _dtype, _heads_3d, _int32, _int32_value, _launch, _on, _table_2d

__all__ = ["attend_shared", "attend_weights", "cache_evict", "MAX_LONG_REQUESTS"]

MAX_LONG_REQUESTS = 8192

EXPORTED_SYMBOLS = ("attend_shared", "attend_shared_workspace", "attend_weights", "cache_evict", "cache_evict_workspace", "gvr_long_status_string")


def _declare(lib):
    i64, i32, p, f32, sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    cache = ctypes.POINTER(_Cache)
    lib.attend_shared.argtypes = [cache, p, i64, i64, i32, i64, i32, p, i64, i64, p, i32, i32, p, p, i64, f32, p, p, p, sz, p]
    lib.attend_shared_workspace.argtypes = [i32, i32, i64, i32, i32, i64, ctypes.POINTER(sz)]
    lib.attend_weights.argtypes = [cache, p, i64, i64, i32, i64, i32, p, i64, i64, p, i32, i32, p, f32, p, i64, p]
    lib.cache_evict.argtypes = [cache, p, i64, p, i64, i64, p, i64, i32, p, i64, i32, i32, p, p, p, i64, p, p, sz, p]
    lib.cache_evict_workspace.argtypes = [i64, i32, ctypes.POINTER(sz)]
    for name in EXPORTED_SYMBOLS[:-1]:
        getattr(lib, name).restype = ctypes.c_int
    lib.gvr_long_status_string.argtypes = [ctypes.c_int]
    lib.gvr_long_status_string.restype = ctypes.c_char_p


def _check(lib, status: int):
    if status != 0:
        from . import GvrError
        raise GvrError(status, lib.gvr_long_status_string(status).decode())


def _call(device: int, call, *args):
    _launch(device, lambda *a: _check(_c._library(), call(*a)) or 0, *args)


def _fp32(t, device: int, name, shape):
    import torch
    _on(t, device, name)
    if t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {shape}")
    return t.data_ptr()


def _weights_2d(t, device: int, requests, least):
    """(address, stride) of fp32 weights [>= requests, >= least]."""
    import torch
    _on(t, device, "weights")
    if t.dtype != torch.float32:
        raise TypeError("weights must be float32")
    shape = t.shape
    if len(shape) != 2 or shape[0] < requests or shape[1] < least or (t.numel() > 0 and shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"weights must be [>= {requests}, >= {least}] (an entry for each place of block_table) with unit inner stride")
    return t.data_ptr(), (t.stride(0) if shape[0] > 1 else shape[1])


def attend_shared(q, cache, block_table, kv_lens, next_n: int, compress_ratio: int, group_starts, prefix_entries, *, scale=None,
                  k_scale: float = 1.0, v_scale: float = 1.0, out=None, lse=None, want_lse: bool = False, stream=None):
    """:func:`attend_decode` over whole caches, without indices, for requests that share prefixes; returns (out, lse or None).

    ``group_starts`` (int32 [groups + 1]) cuts the requests into groups: group g is requests group_starts[g] up to
    group_starts[g + 1].  The first ``prefix_entries[g]`` entries (int32 [groups]) of all its requests are the same, as
    they are behind one prompt, and each request's table has them: they are read once for the whole group, where the
    tables are wide and the requests many enough for that to pay.  The result is that of ``attend_decode``.
    """
    if stream is not None:
        with _current(stream, q):
            return attend_shared(q, cache, block_table, kv_lens, next_n, compress_ratio, group_starts, prefix_entries, scale=scale,
                                 k_scale=k_scale, v_scale=v_scale, out=out, lse=lse, want_lse=want_lse)
    done = (_c._native or _c._short()).attend_shared(q, cache, k_scale, v_scale, scale, out, lse, want_lse, block_table, kv_lens,
                                                     next_n, compress_ratio, group_starts, prefix_entries)
    if done is not None:
        return done
    import torch
    next_n, compress_ratio = _int32_value(next_n, "next_n"), _int32_value(compress_ratio, "compress_ratio")
    device, head, scale, out, lse = _attend(q, cache, k_scale, v_scale, scale, out, lse, want_lse)
    c, rows, heads = head[0], head[5], head[6]
    requests = (rows + next_n - 1) // max(next_n, 1)
    table, table_stride, width = _table_2d(block_table, device, requests)
    lens = _int32(kv_lens, device, "kv_lens", requests)
    prefix = _int32(prefix_entries, device, "prefix_entries")
    groups = prefix_entries.shape[0]
    starts = _int32(group_starts, device, "group_starts", groups + 1 if groups else 0)
    lib, size = _c._library(), ctypes.c_size_t(0)
    with torch.cuda.device(device):  # as many pieces as it has SMs
        _check(lib, lib.attend_shared_workspace(c.num_kv_heads, c.head_dim, rows, heads, next_n, groups, ctypes.byref(size)))
    space = torch.empty(size.value, dtype=torch.uint8, device=q.device)
    _call(device, lib.attend_shared, *head, table, table_stride, width, lens, next_n, compress_ratio, starts, prefix, groups, scale,
          out.data_ptr(), None if lse is None else lse.data_ptr(), space.data_ptr(), size.value)
    return out, lse


def _rows(q, cache, k_scale, v_scale, scale):
    """What attend_weights checks of queries and cache: (device, arguments, scale)."""
    c = _cache_struct(cache, k_scale, v_scale)
    device = cache.get_device()
    _on(q, device, "q")
    kind = _dtype(q, "q")
    row, head = _heads_3d(q, "q", c.head_dim)
    rows, heads, dim = q.shape
    if heads == 0 or heads % c.num_kv_heads:
        raise ValueError(f"q has {heads} heads, no multiple of the cache's {c.num_kv_heads}")
    return device, (c, q.data_ptr(), row, head, kind, rows, heads), 1.0 / math.sqrt(dim) if scale is None else scale


def attend_weights(q, cache, block_table, kv_lens, next_n: int, compress_ratio: int, lse, weights=None, *, scale=None,
                   k_scale: float = 1.0, stream=None):
    """Add to ``weights`` (fp32 [requests, >= pages * page_size]) the attention weight that each entry draws in this step, and return it.

    The arguments up to ``compress_ratio``, ``scale`` and ``k_scale`` are those of an :func:`attend_decode` without
    indices, and ``lse`` (fp32 [rows, heads]) the one that it returned: entry e of request b gets the sum of
    exp(scale * q . k_e - lse) over the request's rows that see it and all their heads.  Entries that no row sees stay as
    they are; without ``weights`` the sums start from zeros.
    """
    if stream is not None:
        with _current(stream, q):
            return attend_weights(q, cache, block_table, kv_lens, next_n, compress_ratio, lse, weights, scale=scale, k_scale=k_scale)
    if weights is not None:
        if (_c._native or _c._short()).attend_weights(q, cache, k_scale, scale, block_table, kv_lens, next_n, compress_ratio, lse, weights):
            return weights
    import torch
    next_n, compress_ratio = _int32_value(next_n, "next_n"), _int32_value(compress_ratio, "compress_ratio")
    device, head, scale = _rows(q, cache, k_scale, 1.0, scale)
    rows, heads = head[5:]
    requests = (rows + next_n - 1) // max(next_n, 1)
    table, table_stride, width = _table_2d(block_table, device, requests)
    lens = _int32(kv_lens, device, "kv_lens", requests)
    sums = _fp32(lse, device, "lse", (rows, heads))
    least = width * cache.shape[1]
    if weights is None:
        weights = torch.zeros((requests, least), dtype=torch.float32, device=q.device)
    to, stride = _weights_2d(weights, device, requests, least)
    _call(device, _c._library().attend_weights, *head, table, table_stride, width, lens, next_n, compress_ratio, sums, scale, to, stride)
    return weights


def cache_evict(weights, cache, block_table, kv_lens, free_pages, keep: int, recent: int, compress_ratio: int = 1, max_released: int | None = None,
                kept=None, new_lens=None, released=None, counts=None, *, stream=None):
    """Cut each request's cache to ``keep`` entries: its ``recent`` last ones, and of the others those of largest weight.

    ``weights`` is fp32 [requests, >= pages * page_size] (as :func:`attend_weights` adds them up; equal ones: the lower
    number stays), ``kv_lens`` int32 [requests] the uncompressed lengths.  Requests of at most ``keep`` entries stay as
    they are.  The kept entries keep their order and become entries 0 .. keep - 1; from the first page that changes they
    are copied to pages taken from ``free_pages`` (int32), so that no page that another request may hold is
    written.  ``block_table`` and ``weights`` are rewritten in place.  Returns ``kept`` (int32 [requests, keep]: the entries' old numbers, -1
    behind them), ``new_lens`` (int32 [requests]), ``released`` (int32 [max_released]: the pages given up, -1 behind
    them) and ``counts`` (int32 [3]: pages taken, pages released, requests left as they were for want of pages, whose row of
    ``kept`` is -1).  Without ``max_released`` the list holds as many as ``released`` does where that is given, else every page
    of the table; a shorter one loses the numbers of those that it has no room for.
    """
    if stream is not None:
        with _current(stream, cache):
            return cache_evict(weights, cache, block_table, kv_lens, free_pages, keep, recent, compress_ratio, max_released, kept, new_lens,
                               released, counts)
    done = (_c._native or _c._short()).cache_evict(weights, cache, block_table, kv_lens, free_pages, keep, recent, compress_ratio,
                                                   max_released, kept, new_lens, released, counts)
    if done is not None:
        return done
    import torch
    keep, recent, compress_ratio = _int32_value(keep, "keep"), _int32_value(recent, "recent"), _int32_value(compress_ratio, "compress_ratio")
    if keep < 1 or not 0 <= recent <= keep or (max_released is not None and max_released < 0):
        raise ValueError(f"keep must be at least 1, recent 0 to keep and max_released at least 0: got {keep}, {recent} and {max_released}")
    c = _cache_struct(cache, 1.0, 1.0)
    device = cache.get_device()
    lens = _int32(kv_lens, device, "kv_lens")
    requests = kv_lens.shape[0]
    table, table_stride, width = _table_2d(block_table, device, requests)
    w, w_stride = _weights_2d(weights, device, requests, width * cache.shape[1])
    free = _int32(free_pages, device, "free_pages")
    if max_released is None:
        max_released = requests * width if released is None else released.numel()

    def ints(t, name, *shape):
        if t is None:
            return torch.empty(shape, dtype=torch.int32, device=cache.device)
        _on(t, device, name)
        if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape}")
        return t

    lib, size = _c._library(), ctypes.c_size_t(0)
    _check(lib, lib.cache_evict_workspace(requests, keep, ctypes.byref(size)))
    kept, new_lens = ints(kept, "kept", requests, keep), ints(new_lens, "new_lens", requests)
    released, counts = ints(released, "released", max_released), ints(counts, "counts", 3)
    space = torch.empty(size.value, dtype=torch.uint8, device=cache.device)
    _call(device, lib.cache_evict, c, w, w_stride, table, table_stride, width, lens, requests, compress_ratio, free, free_pages.shape[0],
          keep, recent, kept.data_ptr(), new_lens.data_ptr(), released.data_ptr(), max_released, counts.data_ptr(), space.data_ptr(), size.value)
    return kept, new_lens, released, counts
