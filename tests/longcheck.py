"""Plain implementations, on the host, of what include/gvr_long.h defines: sums in 64 bits over
requests, rows and heads, and eviction entry by entry.  For small sizes."""
from __future__ import annotations

import numpy as np

import cachecheck


def weights(q, cache, table, lens, next_n, cr, lse, scale, before, k_scale=1.0):
    """(weights after the step, how far fp32 may be off)."""
    rows, heads, dim = q.shape
    pages, ps, hk = cache.shape[:3]
    after, tol = before.astype(np.float64), np.zeros(before.shape)
    seen = cachecheck.row_entries(lens, next_n, cr, rows, table.shape[1] * ps if pages else 0)
    k_all, _ = cachecheck.unpack(cache, dim, k_scale)
    for b in range(-(-rows // next_n)):
        own = range(b * next_n, min((b + 1) * next_n, rows))
        n = max(seen[r] for r in own) if len(own) == next_n else cachecheck.row_entries(lens[b:b + 1], next_n, cr, next_n, table.shape[1] * ps if pages else 0)[-1]
        e = np.arange(n)
        page = table[b, e // ps].astype(np.int64) if n else e
        ok = (page >= 0) & (page < pages)
        drawn, worst = np.zeros(n), np.zeros(n)
        for r in own:
            at = np.flatnonzero(ok & (e < seen[r]))
            for h in range(heads):
                k, x = k_all[page[at], e[at] % ps, h // (heads // hk)], q[r, h].astype(np.float64)
                s = scale * (k @ x)
                p = np.exp(s - np.float64(lse[r, h]))
                size = abs(scale) * (np.abs(k) @ np.abs(x))
                # fp32 products and sums of dim terms, each off by a step of sum |q||k|; score, factor and log-sum
                # in log2 units, rounded at each of four places; the exponential
                off = size * (dim + 8) * 2.0 ** -23 + (size + abs(float(lse[r, h]))) * 2.0 ** -22 + 2.0 ** -21
                drawn[at] += p
                worst[at] += p * off
        after[b, :n] += drawn
        # sums of all rows' heads, each addition half a step of the sum so far; the last one of what was there, too
        tol[b, :n] = worst * 1.01 + (len(own) * heads + 32) * 2.0 ** -24 * drawn + 2.0 ** -24 * np.abs(after[b, :n]) * 1.01
    return after, tol


def chosen(w, n, keep, recent):
    """The old numbers of the entries that stay, ascending: sorted by key, a NaN first, ties by number."""
    older = range(n - recent)
    order = sorted(older, key=lambda i: (0 if np.isnan(w[i]) else 1, 0 if np.isnan(w[i]) else -float(w[i]), i))
    return sorted(order[:keep - recent]) + list(range(n - recent, n))


def evict(w, cache, table, lens, cr, free, keep, recent, max_released):
    """(weights, cache, table, kept, new_lens, released, counts) after the cut; the inputs stay as they are."""
    w, cache, table = w.copy(), cache.copy(), table.copy()
    pages, ps = cache.shape[:2]
    capacity = table.shape[1] * ps if pages else 0
    kept, new, released, taken, left, wanted = np.full((len(lens), keep), -1, np.int32), np.array(lens, np.int32), [], 0, 0, 0
    for r in range(len(lens)):
        n = min(max(int(lens[r]), 0) // cr, capacity)
        if n <= keep:
            kept[r, :n] = np.arange(n)
            continue
        have = -(-n // ps)
        if any(not 0 <= table[r, b] < pages for b in range(have)):
            left += 1
            continue
        stay = chosen(w[r], n, keep, recent)
        first = next((i for i in range(keep) if stay[i] != i), keep) // ps
        need = -(-keep // ps) - first
        wanted += need
        if wanted > len(free):
            left += 1
            continue
        fresh = free[wanted - need:wanted]
        old = table[r, :have].copy()
        for i in range(first * ps, keep):
            if 0 <= fresh[i // ps - first] < pages:
                cache[fresh[i // ps - first], i % ps] = cache[old[stay[i] // ps], stay[i] % ps]
        table[r, first:have] = -1
        table[r, first:first + need] = fresh
        released += list(old[first:])
        taken += need
        kept[r] = stay
        w[r, :keep] = w[r, stay]
        w[r, keep:n] = 0
        new[r] = keep * cr + int(lens[r]) % cr
    out = np.full(max_released, -1, np.int32)
    out[:min(len(released), max_released)] = released[:max_released]
    return w, cache, table, kept, new, out, np.array([taken, len(released), left], np.int32)
