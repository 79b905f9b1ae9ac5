"""Cases for measuring what long-lived requests need of the 4-bit paged cache.

Three operators, each in a plain form (elementary torch operations) and through the package's public
calls (``own``):

* ``shared``  -- attention of decode rows whose requests share long prefixes, each prefix read once for all
  of its requests (``attend_shared``);
* ``weights`` -- the attention weight that each cached entry draws, added up over a step's rows and heads
  (``attend_weights``);
* ``evict``   -- each request's cache cut to its heaviest and its latest entries: which ones, and their rows
  moved together into pages of their own (``cache_evict``).

The cache: uint8 [pages, page_size, kv_heads, row].  A row holds, for one entry and one KV head of
``dim`` values, K codes (dim / 2 bytes, two e2m1 codes per byte, even value in the low half), V
codes (dim / 2), K scales (dim / 16 bytes, e4m3, one per 16 values) and V scales (dim / 16), padded
to 16 bytes.  A value is code * scale.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # Two requests behind one short prefix: the smallest call, where latency counts.
        {"name": "shared_pair", "op": "shared", "requests": 2, "groups": 1, "next_n": 1, "cr": 1, "prefix_lo": 700, "prefix_hi": 700,
         "lo": 1, "hi": 100, "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16", "page_size": 64},
        # The decode batch workload behind one system prompt: 64 requests x 2 rows.
        {"name": "shared_batch", "op": "shared", "requests": 64, "groups": 1, "next_n": 2, "cr": 4, "prefix_lo": 32000,
         "prefix_hi": 32000, "lo": 10, "hi": 2000, "heads": 64, "kv_heads": 8, "dim": 128, "dtype": "bf16", "page_size": 64},
        # Several prompts with their samples, groups of uneven size (one of a single request), odd group of six
        # heads, draft tokens, an idle request.
        {"name": "shared_groups", "op": "shared", "requests": 49, "groups": 7, "next_n": 2, "cr": 1, "prefix_lo": 333,
         "prefix_hi": 12001, "lo": 1, "hi": 1500, "heads": 24, "kv_heads": 4, "dim": 64, "dtype": "f16", "page_size": 16},
        # One KV head shared by 40 query heads, one long document asked 16 times.
        {"name": "shared_document", "op": "shared", "requests": 16, "groups": 1, "next_n": 1, "cr": 1, "prefix_lo": 131071,
         "prefix_hi": 131071, "lo": 20, "hi": 600, "heads": 40, "kv_heads": 1, "dim": 128, "dtype": "f16", "page_size": 32},
        # Wide heads, three prompts.
        {"name": "shared_wide", "op": "shared", "requests": 27, "groups": 3, "next_n": 1, "cr": 1, "prefix_lo": 9001,
         "prefix_hi": 20011, "lo": 100, "hi": 900, "heads": 16, "kv_heads": 2, "dim": 256, "dtype": "bf16", "page_size": 32},
        # One decode row's weights over 8192 entries.
        {"name": "weights_one_row", "op": "weights", "requests": 1, "next_n": 1, "cr": 1, "lo": 8192, "hi": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page_size": 64},
        # A decode batch's weights, an idle request.
        {"name": "weights_batch", "op": "weights", "requests": 64, "next_n": 1, "cr": 1, "lo": 500, "hi": 16384, "heads": 64,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page_size": 64},
        # The last 16 rows of prompts as observers of all of their entries, odd group of six, small heads.
        {"name": "weights_window", "op": "weights", "requests": 19, "next_n": 16, "cr": 1, "lo": 16, "hi": 12345, "heads": 24,
         "kv_heads": 4, "dim": 64, "dtype": "f16", "page_size": 16},
        # One request cut from 9000 entries to 2048.
        {"name": "evict_one", "op": "evict", "requests": 1, "cr": 1, "lo": 9000, "hi": 9000, "keep": 2048, "recent": 256,
         "kv_heads": 8, "dim": 128, "page_size": 64, "sinks": 4},
        # A batch cut to 4096 entries each, most of them a little over it, as after some steps' growth.
        {"name": "evict_batch", "op": "evict", "requests": 64, "cr": 4, "lo": 3900, "hi": 5200, "keep": 4096, "recent": 1000,
         "kv_heads": 8, "dim": 128, "page_size": 64, "sinks": 130},
        # Many short requests, small pages and heads, an odd budget; half of them have nothing to give up.
        {"name": "evict_short", "op": "evict", "requests": 230, "cr": 1, "lo": 1, "hi": 1400, "keep": 701, "recent": 64,
         "kv_heads": 4, "dim": 64, "page_size": 16, "sinks": 0},
        # Long prompts cut to a quarter after their prefill, wide heads.
        {"name": "evict_long", "op": "evict", "requests": 5, "cr": 1, "lo": 60000, "hi": 131072, "keep": 20000, "recent": 4000,
         "kv_heads": 2, "dim": 256, "page_size": 32, "sinks": 1000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "weights", "evict"])
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    common = {"kv_heads": kv_heads, "dim": dim, "page_size": rng.choice([16, 32, 64, 128]), "cr": rng.choice([1, 1, 4])}
    per = kv_heads * dim
    if op == "evict":
        requests = _log(rng, 1, 230)
        keep = _log(rng, 64, max(64, min(20000, 64 * 4096 * 1024 // (requests * per))))
        hi = max(keep + 1, min(131072, int(keep * rng.uniform(1.05, 5))))
        return {"op": op, "requests": requests, "lo": rng.randrange(1, hi), "hi": hi, "keep": keep, "recent": rng.randrange(0, keep * 3 // 4 + 1),
                "sinks": rng.choice([0, 4, keep // 4]), **common}
    common["dtype"] = rng.choice(["bf16", "f16"])
    group = rng.choice([1, 2, 4, 5, 6, 8, 16])
    common["heads"] = kv_heads * group
    if op == "weights":
        next_n, requests = rng.choice([1, 1, 2, 16]), _log(rng, 1, 64)
        # not more products than the listed batch has
        most = min(131072, 64 * 16384 * 1024 // (requests * per), 64 * 16384 * 64 * 128 // (requests * next_n * group * per))
        hi = _log(rng, 100, max(200, most))
        return {"op": op, "requests": requests, "next_n": next_n, "lo": max(1, hi // 30), "hi": hi, **common}
    next_n, requests = rng.choice([1, 1, 2, 3]), _log(rng, 2, 64)
    groups = _log(rng, 1, max(1, requests // 3))
    rows = requests * next_n
    most = min(131071, 128 * 32000 * 64 * 128 // (rows * group * per), 64 * 34000 * 1024 // (requests * per))
    prefix = _log(rng, 60, max(100, most))
    hi = _log(rng, 2, min(2000, max(4, prefix)))
    return {"op": op, "requests": requests, "groups": groups, "next_n": next_n, "prefix_lo": max(1, prefix // rng.choice([1, 2, 8])),
            "prefix_hi": prefix, "lo": 1, "hi": hi, **common}


# -------------------------------------------------------------------- what both sides are given
def _row_bytes(dim):
    return (dim + dim // 8 + 15) // 16 * 16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randint(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _pack(k, v):
    """Rows [n, heads, row] of the cache from K and V [n, heads, dim]: blocks of 16, e4m3 scales, e2m1 codes."""
    codes, scales = [], []
    for x in (k, v):
        b = x.float().unflatten(-1, (-1, 16))
        s = (b.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        q = torch.where(s.float() > 0, b / s.float(), torch.zeros_like(b))
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
        c = (torch.bucketize(q.abs(), edges) + 8 * (q < 0)).flatten(-2)
        codes.append((c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8))
        scales.append(s.squeeze(-1).view(torch.uint8))
    dim = k.shape[-1]
    pad = _row_bytes(dim) - dim - dim // 8
    return torch.cat((*codes, *scales, torch.zeros(*k.shape[:-1], pad, dtype=torch.uint8, device=k.device)), dim=-1)


def _values(rows, dim, which, dtype=torch.float32):
    """K (which = 0) or V (1) values [..., dim] of cache rows [..., row]."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=rows.device, dtype=dtype)
    codes = rows[..., which * dim // 2:(which + 1) * dim // 2]
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    s = rows[..., dim + which * dim // 16:dim + (which + 1) * dim // 16].contiguous().view(torch.float8_e4m3fn).to(dtype)
    return (table[c.int()].unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _make_cache(g, pages, ps, heads, dim):
    """A filled cache: entries drawn from a pool of 2048 quantised ones (normal values whose size
    differs from channel to channel), so that gigabytes are made quickly."""
    size = torch.exp(0.5 * torch.randn(2, 1, heads, dim, generator=g, device="cuda"))
    kv = torch.randn(2, 2048, heads, dim, generator=g, device="cuda") * size
    pool = _pack(kv[0], kv[1]).flatten(1)
    at = torch.randint(0, 2048, (pages * ps,), generator=g, device="cuda")
    return pool[at].view(pages, ps, heads, -1)


def _paged(g, ps, first, entries, width, spare):
    """A block table [requests, width] of pages in random order: request q holds pages for entries [first, entries)
    of its own (the places before are -1), and the `spare` page numbers that no one holds."""
    have, need = first // ps, (entries + ps - 1) // ps
    own_pages = (need - have).clamp(min=0)
    total = int(own_pages.sum())
    order = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    start = own_pages.cumsum(0) - own_pages
    col = torch.arange(max(width, 1), device="cuda")
    at = (start[:, None] + col - have[:, None]).clamp(0, max(total - 1, 0))
    table = torch.where((col >= have[:, None]) & (col < need[:, None]), order[at], -1)
    return table.to(torch.int32).contiguous(), order[total:].contiguous()


def _group_starts(case):
    """Groups of growing size: the i-th of G begins at request i (i + 1) / (G (G + 1)) of all."""
    n, groups = case["requests"], case["groups"]
    return [n * i * (i + 1) // (groups * (groups + 1)) for i in range(groups + 1)]


def _shared(g, s):
    case, ps, cr = s["case"], s["case"]["page_size"], s["case"]["cr"]
    n = case["requests"]
    starts = torch.tensor(_group_starts(case), dtype=torch.int32, device="cuda")
    prefix = _randint(g, case["prefix_lo"], case["prefix_hi"], case["groups"])
    group = torch.searchsorted(starts[1:], torch.arange(n, dtype=torch.int32, device="cuda"), right=True)
    shared = prefix[group].long()
    entries = shared + _randint(g, case["lo"], case["hi"], n)
    lens = entries * cr + _randint(g, 0, cr - 1, n)
    if n > 4:
        lens[n // 2] = 0  # an idle request
    width = (case["prefix_hi"] + case["hi"] + ps - 1) // ps
    # full pages of a prefix are the group's; the page in which it ends is each request's own copy
    own_table, spare = _paged(g, ps, shared, entries, width, int((prefix // ps).sum()) + 3)
    full = (prefix // ps).long()
    col = torch.arange(width, device="cuda")
    common = spare[((full.cumsum(0) - full)[:, None] + col).clamp(max=spare.numel() - 1)]
    table = torch.where(col < (shared // ps)[:, None], common[group], own_table).contiguous()
    cache = _make_cache(g, int(own_table.max()) + 1 if spare.numel() == 0 else int(max(own_table.max(), spare.max())) + 1, ps,
                        case["kv_heads"], case["dim"])
    # what the copies hold of the prefix is the same: the group's first request's
    lead = starts[group].long()
    page, lead_page = table.gather(1, (shared // ps)[:, None])[:, 0].long(), table[lead, shared // ps].long()
    off = torch.arange(ps, device="cuda")
    rows = torch.where((off < (shared % ps)[:, None])[..., None, None], cache[lead_page], cache[page])
    cache[page] = rows
    s.update(cache=cache, table=table, lens=lens.to(torch.int32), starts=starts, prefix=prefix)


def _entries_of_rows(case, lens, cap):
    r = torch.arange(case["requests"] * case["next_n"], device="cuda")
    m = lens[r // case["next_n"]].long()
    n = (m - case["next_n"] + r % case["next_n"] + 1).div(case["cr"], rounding_mode="floor")
    return torch.where(m < case["next_n"], 0, n.clamp(max=cap)).view(case["requests"], case["next_n"])


def _queries(g, case):
    q = 1.5 * torch.randn(case["requests"] * case["next_n"], case["heads"], case["dim"], generator=g, device="cuda")
    return q.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    n, ps, cr = case["requests"], case["page_size"], case["cr"]
    if case["op"] == "shared":
        _shared(g, s)
        s["q"] = _queries(g, case)
        return s
    entries = _randint(g, case["lo"], case["hi"], n).long()
    width = (case["hi"] + ps - 1) // ps
    if case["op"] == "weights":
        lens = (entries * cr + case["next_n"] - 1).to(torch.int32)
        if n > 4:
            lens[n // 2] = 0
        width = (case["hi"] + case["next_n"] + ps - 1) // ps
        s["table"], _ = _paged(g, ps, 0 * entries, entries + case["next_n"], width, 3)
        s["cache"] = _make_cache(g, int(s["table"].max()) + 4, ps, case["kv_heads"], case["dim"])
        s.update(lens=lens, q=_queries(g, case))
        x, _ = _scores(s, torch.float32)
        s["lse"] = torch.logsumexp(x, dim=-1).flatten(2).flatten(0, 1).contiguous()
        # what earlier steps have added up: a few entries drew most
        old = torch.exp(1.5 * torch.randn(n, width * ps, generator=g, device="cuda"))
        s["weights"] = old * (torch.arange(width * ps, device="cuda") < (lens // cr)[:, None])
        return s
    lens = entries * cr + _randint(g, 0, cr - 1, n)
    s["table"], s["free"] = _paged(g, ps, 0 * entries, entries, width, n * ((case["keep"] + ps - 1) // ps) + 3)
    pages = n * (width + (case["keep"] + ps - 1) // ps) + 3  # whatever the lengths
    s["cache"] = _make_cache(g, pages, ps, case["kv_heads"], case["dim"])
    w = torch.exp(2.0 * torch.randn(n, width * ps, generator=g, device="cuda"))
    # many entries were never looked at: equal weights
    w = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, 0.0, w)
    w[:, :case["sinks"]] += 1e5  # the first entries draw most of all
    s["weights"] = w * (torch.arange(width * ps, device="cuda") < entries[:, None])
    s.update(lens=lens.to(torch.int32), released=n * width)
    return s


# ------------------------------------------------------------------------------- plain forms
def _scores(s, dtype):
    """Scores [requests, next_n, kv_heads, group, entries] and the slots read [requests, entries]; -inf where a row sees nothing."""
    case, ps = s["case"], s["case"]["page_size"]
    hk, d = case["kv_heads"], case["dim"]
    seen = _entries_of_rows(case, s["lens"], s["table"].shape[1] * ps)
    col = torch.arange(max(int(seen.max()), 1), device="cuda")
    page = s["table"][:, col // ps].long()
    slot = torch.where(page >= 0, page * ps + col % ps, 0)
    flat = s["cache"].view(-1, hk, s["cache"].shape[-1])
    k = _values(flat[slot], d, 0, dtype)  # [requests, n, hk, d]
    q = s["q"].to(dtype).view(case["requests"], case["next_n"], hk, -1, d)
    x = torch.einsum("bjhgd,bnhd->bjhgn", q, k) / math.sqrt(d)
    ok = (col < seen[..., None]) & (page >= 0)[:, None]
    return x.masked_fill(~ok[:, :, None, None, :], -math.inf), slot


def _plain_shared(s):
    case = s["case"]
    x, slot = _scores(s, torch.float32)
    v = _values(s["cache"].view(-1, case["kv_heads"], s["cache"].shape[-1])[slot], case["dim"], 1)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bjhgn,bnhd->bjhgd", p, v) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + top).squeeze(-1)
    return o.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(s["q"].shape[:2])


def _plain_weights(s):
    case = s["case"]
    x, _ = _scores(s, torch.float32)
    lse = s["lse"].view(*x.shape[:-1], 1)
    p = torch.where(x == -math.inf, 0.0, torch.exp(x - lse)).sum((1, 2, 3))
    w = s["weights"].clone()
    w[:, :p.shape[1]] += p
    return w


def _plain_evict(s):
    case, ps, cr, keep = s["case"], s["case"]["page_size"], s["case"]["cr"], s["case"]["keep"]
    table, weights, dev = s["table"].clone(), s["weights"].clone(), s["lens"].device
    requests, width = table.shape
    n = s["lens"].long() // cr
    col = torch.arange(weights.shape[1], device=dev)
    cut = n > keep
    # the heaviest of the older entries, ties to the lower number, and the latest ones
    older = (n - case["recent"])[:, None]
    order = torch.where(col < older, weights, -math.inf).sort(dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, col.expand_as(order))
    chosen = ((rank < keep - case["recent"]) & (col < older)) | (col >= older)
    chosen = torch.where(cut[:, None], chosen, True) & (col < n[:, None])
    kept = torch.where(chosen, col, 1 << 30).sort(dim=1).values
    kept = torch.nn.functional.pad(kept, (0, max(0, keep - kept.shape[1])), value=1 << 30)[:, :keep]
    kept = torch.where(kept < 1 << 30, kept, -1)
    # pages whose entries all stay where they are stay; the others are made anew
    at = torch.arange(keep, device=dev)
    stays = ((kept == at) & cut[:, None]).int().cumprod(1).sum(1)
    first = torch.where(cut, stays // ps, (keep + ps - 1) // ps)
    need = torch.where(cut, (keep + ps - 1) // ps - first, 0)
    given = torch.where(cut, (n + ps - 1) // ps - first, 0)
    before, gone = need.cumsum(0) - need, given.cumsum(0) - given
    block = torch.arange(width, device=dev)
    new = cut[:, None] & (block >= first[:, None]) & (block < (first + need)[:, None])
    old = cut[:, None] & (block >= first[:, None]) & (block < (first + given)[:, None])
    pages = s["free"][(before[:, None] + block - first[:, None]).clamp(0, s["free"].numel() - 1)]
    released = torch.full((s["released"],), -1, dtype=torch.int32, device=dev)
    released[(gone[:, None] + block - first[:, None])[old]] = table[old]
    after = torch.where(new, pages, torch.where(old, -1, table))
    moved = cut[:, None] & (at // ps >= first[:, None])
    src = (table.gather(1, (kept.clamp(min=0) // ps)).long() * ps + kept % ps)[moved]
    dst = (after.gather(1, (at // ps).clamp(max=width - 1).expand(requests, keep)).long() * ps + at % ps)[moved]
    flat = s["cache"].view(-1, s["cache"].shape[2] * s["cache"].shape[3])
    flat[dst] = flat[src]
    few = torch.where(col < keep, 1, 0)[None] * weights.gather(1, torch.nn.functional.pad(kept, (0, max(0, weights.shape[1] - keep)))[:, :weights.shape[1]].clamp(min=0))
    weights = torch.where(cut[:, None], few, weights)
    lens = torch.where(cut, keep * cr + s["lens"] % cr, s["lens"]).to(torch.int32)
    counts = torch.stack((need.sum(), given.sum(), 0 * need.sum())).to(torch.int32)
    return kept.to(torch.int32), lens, released, counts, after, weights, s["cache"]


def run(state):
    s, case = state, state["case"]
    if own:
        import sparse_attention_indexer_exact_gb300 as gvr
        if case["op"] == "shared":
            return gvr.attend_shared(s["q"], s["cache"], s["table"], s["lens"], case["next_n"], case["cr"], s["starts"], s["prefix"],
                                     want_lse=True)
        if case["op"] == "weights":
            w = s["weights"].clone()
            return gvr.attend_weights(s["q"], s["cache"], s["table"], s["lens"], case["next_n"], case["cr"], s["lse"], w)
        table, weights = s["table"].clone(), s["weights"].clone()
        kept, lens, released, counts = gvr.cache_evict(weights, s["cache"], table, s["lens"], s["free"], case["keep"], case["recent"],
                                                       case["cr"], s["released"])
        return kept, lens, released, counts, table, weights, s["cache"]
    if case["op"] == "shared":
        return _plain_shared(s)
    return _plain_weights(s) if case["op"] == "weights" else _plain_evict(s)


# --------------------------------------------------------------------------- work and definition
def work(case):
    ps, per = case["page_size"], case["kv_heads"] * case["dim"]
    if case["op"] == "evict":
        lo, hi, keep, row = case["lo"], case["hi"], case["keep"], case["kv_heads"] * _row_bytes(case["dim"])
        over = max(0, hi - max(lo - 1, keep)) / (hi - lo + 1)  # requests that are cut
        n = (max(lo, keep + 1) + hi) / 2  # their entries
        moved = keep - min(keep, case["sinks"]) // ps * ps  # whole pages of first entries stay
        # rows read and written; weights read, and the kept ones written; entry numbers, tables and lists
        each = 2 * moved * row + 4 * n + 4 * n + 4 * keep + 12 * n / ps
        return {"bytes": case["requests"] * (over * each + (1 - over) * 4 * keep + 12) + 4 * case["requests"] * hi / ps, "flops": 0}
    rows, heads = case["requests"] * case["next_n"], case["heads"]
    busy = (case["requests"] - 1) / case["requests"] if case["requests"] > 4 else 1.0
    mean = (case["lo"] + case["hi"]) / 2
    if case["op"] == "weights":
        # K codes and scales once, queries and their log-sums, the weights read and written
        nbytes = case["requests"] * busy * mean * (per * 9 / 16 + 8) + rows * heads * (2 * case["dim"] + 4)
        return {"bytes": nbytes, "flops": 2 * rows * busy * mean * heads * case["dim"]}
    prefix = (case["prefix_lo"] + case["prefix_hi"]) / 2
    reads = (case["groups"] * prefix + case["requests"] * busy * mean) * per * 9 / 8
    return {"bytes": reads + rows * heads * (4 * case["dim"] + 4), "flops": 4 * rows * busy * (prefix + mean) * heads * case["dim"]}


def _exact_evict(s):
    """The weights alone: all else is whole numbers."""
    case, w = s["case"], s["weights"].double().cpu().numpy()
    for b, length in enumerate(s["lens"].tolist()):
        n = length // case["cr"]
        if n > case["keep"]:
            older = np.arange(n - case["recent"])
            heavy = np.lexsort((older, -w[b, older]))[:case["keep"] - case["recent"]]
            few = w[b, np.concatenate((np.sort(heavy), np.arange(n - case["recent"], n)))]
            w[b] = 0
            w[b, :case["keep"]] = few
    return None, None, None, None, None, torch.from_numpy(w), None


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    hk, d, ps, rows_of = case["kv_heads"], case["dim"], case["page_size"], case["next_n"]
    signed = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda", dtype=torch.float64)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if case["op"] == "weights" else None
    for b in range(case["requests"]):
        length = int(s["lens"][b])
        e = torch.arange(length // case["cr"] if length >= rows_of else 0, device="cuda")
        if e.numel() == 0:
            continue
        rows = s["cache"][s["table"][b, torch.div(e, ps, rounding_mode="floor")].long(), e % ps].transpose(0, 1)  # [hk, n, row]
        kv = []
        for i in (0, 1):
            codes = rows[..., i * (d // 2):(i + 1) * (d // 2)]
            x = torch.empty(*codes.shape[:-1], d, dtype=torch.float64, device="cuda")
            x[..., 0::2] = signed[(codes % 16).long()]
            x[..., 1::2] = signed[torch.div(codes, 16, rounding_mode="floor").long()]
            scales = rows[..., d + i * (d // 16):d + (i + 1) * (d // 16)].contiguous().view(torch.float8_e4m3fn)
            kv.append(x * scales.double().repeat_interleave(16, dim=-1))
        for j in range(rows_of):
            n, r = (length - rows_of + j + 1) // case["cr"], b * rows_of + j
            if n == 0:
                continue
            x = s["q"][r].double().view(hk, -1, d) @ kv[0][:, :n].transpose(1, 2) / math.sqrt(d)
            if weights is not None:
                weights[b, :n] += torch.exp(x - s["lse"][r].double().view(hk, -1, 1)).sum((0, 1))
            else:
                lse[r] = torch.logsumexp(x, dim=-1).flatten()
                out[r] = (torch.softmax(x, dim=-1) @ kv[1][:, :n]).flatten(0, 1)
    return weights if weights is not None else (out, lse)
