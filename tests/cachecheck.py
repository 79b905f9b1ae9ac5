"""A plain implementation, in 64 bits on the host, of the 4-bit cache and its operators.

Written from the definitions in include/gvr_cache.h: e2m1 codes, e4m3 scales of 16 values, entries
found through block tables, softmax over the entries a row sees.  Loops over requests and rows; for
small sizes.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
ROW_BYTES = {64: 80, 128: 144, 256: 288}


def e4m3_values():
    """The value of each of the 256 codes."""
    v = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            x = np.nan
        v[code] = -x if code & 128 else x
    return v


E4M3 = e4m3_values()


def nearest(x, grid):
    """Index of the grid value nearest to x >= 0, ties to the even index, saturating."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, x, side="left")  # x > mid[i - 1], x <= mid[i]
    tie = (i < mid.size) & (x == mid[np.minimum(i, mid.size - 1)])
    return np.where(tie & (i % 2 == 1), i + 1, i)


def quantise(x, factor):
    """x [..., dim] -> (codes 0..15, scale codes), in 64 bits but for the quotients, which are fp32."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 16)
    nan = np.isnan(b).any(-1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        want = np.minimum(np.abs(b).max(-1, keepdims=True) / np.float32(np.float32(6) * np.float32(factor)), np.float32(448))
    want = np.where(nan, 0, want)
    sc = nearest(want.astype(np.float64), E4M3[:127])
    unit = np.float32(E4M3[sc]) * np.float32(factor)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        q = np.where((unit > 0) & ~nan, b / unit, 0).astype(np.float64)
    code = nearest(np.abs(q), E2M1) + 8 * np.signbit(q)
    code = np.where((unit > 0) & ~nan, code, 0)
    return code.reshape(x.shape).astype(np.int64), np.where(nan, 127, sc)[..., 0]


def dequantise(code, sc, factor):
    c = np.where(code >= 8, -E2M1[code & 7], E2M1[code & 7]).reshape(*code.shape[:-1], -1, 16)
    return (c * E4M3[sc][..., None] * factor).reshape(code.shape)


def unpack(rows, dim, k_scale=1.0, v_scale=1.0):
    """K and V values in 64 bits of cache rows (uint8 [..., row])."""
    got = []
    for i, f in enumerate((k_scale, v_scale)):
        two = rows[..., i * dim // 2:(i + 1) * dim // 2]
        code = np.stack((two & 15, two >> 4), -1).reshape(*two.shape[:-1], dim).astype(np.int64)
        sc = rows[..., dim + i * dim // 16:dim + (i + 1) * dim // 16]
        got.append(dequantise(code, sc, float(np.float32(f))))
    return got


def pack(k, v, k_scale=1.0, v_scale=1.0):
    dim = k.shape[-1]
    rows = np.zeros((*k.shape[:-1], ROW_BYTES[dim]), np.uint8)
    for i, (x, f) in enumerate(((k, k_scale), (v, v_scale))):
        code, sc = quantise(x, f)
        rows[..., i * dim // 2:(i + 1) * dim // 2] = code[..., 0::2] + 16 * code[..., 1::2]
        rows[..., dim + i * dim // 16:dim + (i + 1) * dim // 16] = sc
    return rows


def tables(cached, lens, free, table, max_new, ps, cr):
    """(block table, slots, counts) after a step."""
    table = table.copy()
    width, slots, taken, missing = table.shape[1], [], 0, 0
    for q in range(len(lens)):
        e0, e1 = max(int(cached[q]), 0) // cr, max(int(lens[q]), 0) // cr
        have, want = -(-e0 // ps), -(-e1 // ps)
        missing += max(want - width, 0)
        for b in range(have, min(want, width)):
            if taken < len(free):
                table[q, b] = free[taken]
                taken += 1
            else:
                table[q, b] = -1
                missing += 1
        for e in range(e0, e1):
            page = int(table[q, e // ps]) if e // ps < width else -1
            s = page * ps + e % ps
            slots.append(s if page >= 0 and s < 2 ** 31 - 1 else -1)
    out = np.full(max_new, -1, np.int64)
    out[:min(len(slots), max_new)] = slots[:max_new]
    return table, out, np.array([len(slots), taken, missing])


def row_entries(kv, next_n, cr, rows, cap):
    out = []
    for r in range(rows):
        m = int(kv[r // next_n])
        out.append(0 if m < next_n else min((m - next_n + r % next_n + 1) // cr, cap))
    return out


def attend(q, cache, table, entries, requests, indices, scale, k_scale=1.0, v_scale=1.0):
    """Per row in 64 bits: (out, lse, bound of the sum of p|v|, bound of scale * sum |q||k|, entries).

    ``entries[r]`` / ``requests[r]``: what row r sees; ``indices`` int [rows, k] or None."""
    rows, heads, dim = q.shape
    pages, ps, hk = cache.shape[:3]
    k_all, v_all = unpack(cache, dim, k_scale, v_scale)
    out, lse = np.zeros((rows, heads, dim)), np.full((rows, heads), -np.inf)
    spread, size, used = np.zeros((rows, heads, dim)), np.zeros((rows, heads)), np.zeros(rows, np.int64)
    for r in range(rows):
        e = np.arange(entries[r]) if indices is None else indices[r].astype(np.int64)
        e = e[(e >= 0) & (e < entries[r])]
        if not 0 <= requests[r] < table.shape[0] or e.size == 0:
            continue
        page = table[requests[r], e // ps].astype(np.int64)
        ok = (page >= 0) & (page < pages)
        page, off = page[ok], (e % ps)[ok]
        used[r] = page.size
        if page.size == 0:
            continue
        for h in range(heads):
            g = h // (heads // hk)
            k, v, x = k_all[page, off, g], v_all[page, off, g], q[r, h].astype(np.float64)
            s = scale * (k @ x)
            top = s.max()
            p = np.exp(s - top)
            out[r, h] = p @ v / p.sum()
            lse[r, h] = top + np.log(p.sum())
            spread[r, h] = p @ np.abs(v) / p.sum()
            size[r, h] = abs(scale) * (np.abs(k) @ np.abs(x)).max()
    return out, lse, spread, size, used


def attend_tolerance(ref, eps, v_max):
    """Largest |difference| of (out, lse) that the documented roundings allow, element by element.

    fp32 scores: each of head_dim products and sums is off by at most a step, 2^-23, of sum |q||k|;
    to that the factor's and the exponential's roundings, 2^-21 of the score and 2^-21: a relative
    error `d` of each p.  P to f16: half a step, 2^-11 (below 2^-14 an absolute 2^-25, each p being
    held relative to a maximum of at least 1).  Sums over n entries in fp32: n 2^-24 each for
    numerator and denominator.  The output's own rounding: half a step of its type."""
    out, lse, spread, size, used = ref
    dim = out.shape[-1]
    n = used[:, None]
    d = size * (dim + 8) * 2.0 ** -23 + 2.0 ** -21
    rel = 2.0 ** -11 + 2 * d + 2 * n * 2.0 ** -24
    tol = eps / 2 * np.abs(out) + (1 + eps) * (rel[..., None] * spread + n[..., None] * 2.0 ** -25 * v_max)
    with np.errstate(invalid="ignore"):
        tol_lse = d + (n + 8) * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(lse))
    return tol + 1e-30, np.where(np.isfinite(lse), tol_lse, 0)
