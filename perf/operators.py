"""Cases for measuring the 4-bit paged cache operators beside the top-K selection.

Three operators, each in a plain form (elementary torch operations in 32 bits) and through the
package's public calls (``own``):

* ``tables``  -- block tables and slot maps from request lengths (``cache_tables``);
* ``append``  -- K and V written into the 4-bit paged cache and read back (``cache_append``,
  ``cache_read``);
* ``decode`` / ``prefill`` -- attention over that cache, at the top-K selection's indices or over
  the whole cache (``attend_decode``, ``attend_prefill``).

The cache: uint8 [pages, page_size, kv_heads, row].  A row holds, for one entry and one KV head of
``dim`` values, K codes (dim / 2 bytes, two e2m1 codes per byte, even value in the low half), V
codes (dim / 2), K scales (dim / 16 bytes, e4m3, one per 16 values) and V scales (dim / 16), padded
to 16 bytes.  A value is code * scale * a global factor (a power of two in these cases).
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # One decode step of 64 requests with two draft tokens each, at the lengths of the decode
        # batch workload: at most one new entry per request.
        {"name": "tables_step", "op": "tables", "requests": 64, "page_size": 64, "cr": 4, "lo": 16384, "hi": 524288,
         "new_lo": 2, "new_hi": 2, "width": 2049, "pad": 64},
        # Admission of 230 prompts of 1 to 8192 tokens onto caches of up to 2000 tokens.
        {"name": "tables_prompts", "op": "tables", "requests": 230, "page_size": 16, "cr": 1, "lo": 0, "hi": 2000,
         "new_lo": 1, "new_hi": 8192, "width": 640, "pad": 20000},
        # The 128 new rows of a decode batch with eight small KV heads.
        {"name": "append_step", "op": "append", "tokens": 128, "heads": 8, "dim": 64, "dtype": "f16", "page_size": 32,
         "padded": 5},
        # A prompt chunk of odd length, K and V as slices of one projection, padding rows at the end.
        {"name": "append_prompt", "op": "append", "tokens": 16333, "heads": 8, "dim": 128, "dtype": "bf16",
         "page_size": 64, "padded": 333},
        # One decode row of 8192 entries, 512 selected: the smallest call, where latency counts.
        {"name": "decode_one_row", "op": "decode", "requests": 1, "next_n": 1, "cr": 1, "k": 512, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page_size": 64, "lo": 8192, "hi": 8192},
        # The decode batch workload: 64 requests x 2 rows, 1024 selected of up to 131072 entries.
        {"name": "decode_batch", "op": "decode", "requests": 64, "next_n": 2, "cr": 4, "k": 1024, "heads": 64,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page_size": 64, "lo": 16384, "hi": 524288},
        # One KV head shared by 40 query heads, 2048 selected.
        {"name": "decode_shared_head", "op": "decode", "requests": 37, "next_n": 1, "cr": 1, "k": 2048, "heads": 40,
         "kv_heads": 1, "dim": 128, "dtype": "f16", "page_size": 32, "lo": 1000, "hi": 65536},
        # One long request read whole (the layers that do not select).
        {"name": "whole_one_row", "op": "decode", "requests": 1, "next_n": 1, "cr": 1, "k": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page_size": 64, "lo": 131071, "hi": 131071},
        # A ragged batch read whole, odd group of six, small heads, draft tokens, an idle request.
        {"name": "whole_ragged", "op": "decode", "requests": 48, "next_n": 2, "cr": 1, "k": 0, "heads": 24,
         "kv_heads": 4, "dim": 64, "dtype": "f16", "page_size": 16, "lo": 1, "hi": 16384},
        # Wide heads read whole.
        {"name": "whole_wide", "op": "decode", "requests": 6, "next_n": 1, "cr": 1, "k": 0, "heads": 16, "kv_heads": 2,
         "dim": 256, "dtype": "bf16", "page_size": 32, "lo": 9001, "hi": 20011},
        # Rows of the prefill tile (packed requests of 512 to 8192 tokens), 2048 selected each.
        {"name": "prefill_tile", "op": "prefill", "rows": 700, "k": 2048, "heads": 32, "kv_heads": 4, "dim": 128,
         "dtype": "bf16", "page_size": 64, "longest": 8192},
        # A short chunk over small heads.
        {"name": "prefill_chunk", "op": "prefill", "rows": 97, "k": 512, "heads": 16, "kv_heads": 2, "dim": 64,
         "dtype": "f16", "page_size": 16, "longest": 1536},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "decode", "whole", "prefill"])
    if op == "tables":
        prompt = rng.random() < 0.5
        requests = _log(rng, 1, 230 if prompt else 1500)
        ps, cr = rng.choice([16, 32, 64, 128]), rng.choice([1, 1, 4])
        hi = _log(rng, 100, 20000) if prompt else _log(rng, 2000, 262144)
        new_hi = _log(rng, 1, 8192) if prompt else 4
        return {"op": op, "requests": requests, "page_size": ps, "cr": cr, "lo": 0, "hi": hi, "new_lo": rng.choice([0, 1]),
                "new_hi": new_hi, "width": (hi + new_hi) // cr // ps + rng.choice([1, 2, 7]), "pad": rng.randrange(0, 200)}
    heads_kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    common = {"dim": dim, "dtype": rng.choice(["bf16", "f16"]), "page_size": rng.choice([16, 32, 64, 128])}
    if op == "append":
        tokens = _log(rng, 1, 16333 * 1024 // (heads_kv * dim) if heads_kv * dim > 1024 else 16333)
        return {"op": op, "tokens": tokens, "heads": heads_kv, "padded": rng.randrange(0, tokens // 4 + 1), **common}
    heads = heads_kv * rng.choice([1, 2, 4, 5, 6, 8, 16])
    common.update(heads=heads, kv_heads=heads_kv)
    if op == "prefill":
        k = rng.choice([512, 1024, 2048])
        most = min(700, 700 * 2048 * 512 // (k * heads_kv * dim))
        return {"op": op, "rows": _log(rng, 8, most), "k": k, "longest": _log(rng, 300, 8192), **common}
    next_n, cr = rng.choice([1, 1, 2, 3]), rng.choice([1, 4])
    if op == "decode":
        k = rng.choice([512, 1024, 2048])
        requests = _log(rng, 1, max(1, min(64, 64 * 2 * 1024 * 1024 // (k * next_n * heads_kv * dim))))
        hi = _log(rng, 2000, 131072) * cr
        return {"op": op, "requests": requests, "next_n": next_n, "cr": cr, "k": k, "lo": max(1, hi // 16), "hi": hi, **common}
    requests = _log(rng, 1, 48)
    hi = _log(rng, 100, max(200, min(131072, 131072 * 1024 // (heads_kv * dim * requests)))) * cr
    return {"op": "decode", "requests": requests, "next_n": next_n, "cr": cr, "k": 0, "lo": max(1, hi // 50), "hi": hi, **common}


# -------------------------------------------------------------------- what both sides are given
def _row_bytes(dim):
    return (dim + dim // 8 + 15) // 16 * 16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randint(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _quantise(x, factor):
    """x [..., dim] -> (code values, scales) in fp32: blocks of 16, e4m3 scales, e2m1 codes."""
    b = x.float().unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1, keepdim=True) / (6.0 * factor)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    q = torch.where(s > 0, b / (s * factor), torch.zeros_like(b))
    a = q.abs()
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int()
         + (a > 5.0).int())
    code = c + 8 * (q < 0).int()
    return code.flatten(-2), s.squeeze(-1)


def _pack(k, v, factors):
    """Rows [n, heads, row] of the cache from K and V [n, heads, dim]."""
    dim = k.shape[-1]
    (kc, ks), (vc, vs) = _quantise(k, factors[0]), _quantise(v, factors[1])
    two = [c[..., 0::2] + 16 * c[..., 1::2] for c in (kc, vc)]
    parts = [t.to(torch.uint8) for t in two] + [s.to(torch.float8_e4m3fn).view(torch.uint8) for s in (ks, vs)]
    pad = _row_bytes(dim) - dim - dim // 8
    if pad:
        parts.append(torch.zeros(*k.shape[:-1], pad, dtype=torch.uint8, device=k.device))
    return torch.cat(parts, dim=-1)


def _unpack(rows, dim, factors, dtype=torch.float32):
    """K and V values [..., dim] of cache rows [..., row]."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=rows.device, dtype=dtype)
    got = []
    for i in (0, 1):
        codes = rows[..., i * dim // 2:(i + 1) * dim // 2]
        c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
        s = rows[..., dim + i * dim // 16:dim + (i + 1) * dim // 16].contiguous().view(torch.float8_e4m3fn).to(dtype)
        x = table[c.long()].unflatten(-1, (-1, 16)) * (s * factors[i]).unsqueeze(-1)
        got.append(x.flatten(-2))
    return got


def _make_cache(g, pages, ps, heads, dim):
    """A filled cache: entries drawn from a pool of 2048 quantised ones (normal values whose size
    differs from channel to channel), so that gigabytes are made quickly."""
    size = torch.exp(0.5 * torch.randn(2, 1, heads, dim, generator=g, device="cuda"))
    kv = torch.randn(2, 2048, heads, dim, generator=g, device="cuda") * size
    pool = _pack(kv[0], kv[1], (1.0, 1.0)).flatten(1)
    at = torch.randint(0, 2048, (pages * ps,), generator=g, device="cuda")
    return pool[at].view(pages, ps, heads, -1)


def _select(g, n, k):
    """Index rows as the selection writes them: k distinct entries below n in no order, or the
    identity and -1 where n <= k."""
    rows = n.numel()
    top = max(int(n.max()), k, 1)
    score = torch.rand(rows, top, generator=g, device="cuda")
    col = torch.arange(top, device="cuda")
    score.masked_fill_(col >= n[:, None], -1.0)
    idx = score.topk(k, dim=1, sorted=False).indices
    col = col[:k]
    idx = torch.where((n <= k)[:, None], torch.where(col < n[:, None], col, -1), idx)
    return idx.to(torch.int32)


def _row_entries(case, kv, cap):
    """Valid entries of each decode row."""
    r = torch.arange(case["requests"] * case["next_n"], device="cuda")
    m = kv[r // case["next_n"]].long()
    n = (m - case["next_n"] + r % case["next_n"] + 1).div(case["cr"], rounding_mode="floor")
    return torch.where(m < case["next_n"], 0, n.clamp(max=cap))


def _paged(g, case, entries, heads):
    """A cache whose pages lie in random order and the block table that finds them."""
    ps = case["page_size"]
    width = (int(entries.max()) + ps - 1) // ps
    need = (entries + ps - 1) // ps
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    first = need.cumsum(0) - need
    col = torch.arange(max(width, 1), device="cuda")
    table = torch.where(col < need[:, None], order[(first[:, None] + col).clamp(max=pages - 1)], -1)
    return _make_cache(g, pages, ps, heads, case["dim"]), table.to(torch.int32).contiguous()


def _slot_room(case):
    """Slots of the map: room for the step's most new entries, and some more."""
    return case["requests"] * (case["new_hi"] // case["cr"] + 1) + case["pad"]


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "tables":
        n, ps, cr = case["requests"], case["page_size"], case["cr"]
        cached = _randint(g, case["lo"], case["hi"], n)
        lens = cached + _randint(g, case["new_lo"], case["new_hi"], n)
        have = (cached // cr + ps - 1) // ps
        need = (lens // cr + ps - 1) // ps
        total = int(need.sum())
        order = torch.randperm(total + 5, generator=g, device="cuda").to(torch.int32)
        first = have.cumsum(0) - have
        col = torch.arange(case["width"], device="cuda")
        table = torch.where(col < have[:, None], order[(first[:, None] + col).clamp(max=total)], -1).to(torch.int32)
        s.update(cached=cached, lens=lens, table=table.contiguous(), free=order[int(have.sum()):].contiguous(),
                 new=_slot_room(case))
    elif case["op"] == "append":
        n, h, d, ps = case["tokens"], case["heads"], case["dim"], case["page_size"]
        qkv = torch.randn(n, 3 * h, d, generator=g, device="cuda") * torch.exp(torch.randn(3 * h, d, generator=g, device="cuda"))
        qkv = qkv.to(DTYPES[case["dtype"]])
        pages = (n + ps - 1) // ps + 7
        slots = torch.randperm(pages, generator=g, device="cuda")[:, None] * ps + torch.arange(ps, device="cuda")
        slots = slots.flatten()[:n].to(torch.int32)
        slots[n - case["padded"]:] = -1
        cache = torch.zeros(pages, ps, h, _row_bytes(d), dtype=torch.uint8, device="cuda")
        s.update(k=qkv[:, h:2 * h], v=qkv[:, 2 * h:], slots=slots.contiguous(), cache=cache)
    else:
        dt = DTYPES[case["dtype"]]
        if case["op"] == "decode":
            kv = _randint(g, case["lo"], case["hi"], case["requests"])
            if case["requests"] > 4:
                kv[case["requests"] // 2] = 0  # an idle request
            cap = case["hi"] // case["cr"]
            n = _row_entries(case, kv, cap)
            s["cache"], s["table"] = _paged(g, case, kv // case["cr"], case["kv_heads"])
            s.update(lens=kv)
        else:
            # packed requests of (1, 3, 8, 16) sixteenths of the longest; rows spread over their positions
            lengths = torch.tensor([max(1, case["longest"] * p // 16) for p in (1, 3, 8, 16)], device="cuda")
            start = lengths.cumsum(0) - lengths
            at = torch.arange(case["rows"], device="cuda") * int(lengths.sum()) // case["rows"]
            req = torch.searchsorted(lengths.cumsum(0), at, right=True)
            n = at - start[req] + 1
            s["cache"], s["table"] = _paged(g, case, lengths, case["kv_heads"])
            s.update(requests=req.to(torch.int32), starts=start[req].to(torch.int32), ends=(start[req] + n).to(torch.int32))
        if case["k"]:
            s["indices"] = _select(g, n, case["k"])
        rows = n.numel()
        q = torch.randn(rows, case["heads"], case["dim"], generator=g, device="cuda")
        s["q"] = (1.5 * q).to(dt)
    return s


# ------------------------------------------------------------------------------- plain forms
def _plain_tables(s):
    case, ps, cr = s["case"], s["case"]["page_size"], s["case"]["cr"]
    e0, e1 = s["cached"].long() // cr, s["lens"].long() // cr
    width, new = case["width"], s["new"]
    have = (e0 + ps - 1) // ps
    need = ((e1 + ps - 1) // ps).clamp(max=width)
    pages, count = (need - have).clamp(min=0), (e1 - e0).clamp(min=0)
    first, end = pages.cumsum(0) - pages, count.cumsum(0)
    col = torch.arange(width, device=e0.device)
    j = first[:, None] + col - have[:, None]
    given = torch.where(j < s["free"].numel(), s["free"][j.clamp(0, s["free"].numel() - 1)], -1)
    table = torch.where((col >= have[:, None]) & (col < need[:, None]), given, s["table"])
    t = torch.arange(new, device=e0.device)
    r = torch.searchsorted(end, t, right=True).clamp(max=end.numel() - 1)
    p = e0[r] + t - (end - count)[r]
    block = (p // ps).clamp(0, width - 1)
    page = table[r, block].long()
    ok = (t < end[-1]) & (p // ps < width) & (page >= 0)
    slots = torch.where(ok, page * ps + p % ps, -1).to(torch.int32)
    taken = pages.sum().clamp(max=s["free"].numel())
    short = (((e1 + ps - 1) // ps - need).clamp(min=0)).sum() + pages.sum() - taken
    return table, slots, torch.stack((end[-1], taken, short)).to(torch.int32)


def _plain_append(s):
    case = s["case"]
    flat = s["cache"].view(-1, case["heads"], s["cache"].shape[-1])
    ok = s["slots"] >= 0
    flat[s["slots"][ok].long()] = _pack(s["k"][ok], s["v"][ok], (1.0, 0.5))
    k, v = _unpack(flat[s["slots"].clamp(min=0).long()], case["dim"], (1.0, 0.5))
    dt = s["k"].dtype
    return (k * ok[:, None, None]).to(dt), (v * ok[:, None, None]).to(dt)


def _entries(s):
    """Request, entries and (padded) entry numbers of every row, from what the caller has."""
    case = s["case"]
    cap = s["table"].shape[1] * case["page_size"]
    if case["op"] == "decode":
        n = _row_entries(case, s["lens"], cap)
        req = torch.arange(n.numel(), device="cuda") // case["next_n"]
    else:
        req = s["requests"].long()
        n = (s["ends"] - s["starts"]).long().clamp(0, cap)
    if case["k"]:
        idx = s["indices"].long()
    else:
        idx = torch.arange(cap, device="cuda").expand(n.numel(), cap)
    ok = (idx >= 0) & (idx < n[:, None])
    at = torch.where(ok, idx, 0)
    slot = s["table"][req[:, None], at // case["page_size"]].long() * case["page_size"] + at % case["page_size"]
    return torch.where(ok, slot, 0), ok


def _attend(s, dtype):
    case = s["case"]
    hk, d = case["kv_heads"], case["dim"]
    slot, ok = _entries(s)
    q = s["q"].to(dtype).unflatten(1, (hk, -1))
    flat = s["cache"].view(-1, hk, s["cache"].shape[-1])
    k, v = _unpack(flat[slot], d, (1.0, 1.0), dtype)  # [rows, n, hk, d]
    x = torch.einsum("rhgd,rnhd->rhgn", q, k) / math.sqrt(d)
    x = x.masked_fill(~ok[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("rhgn,rnhd->rhgd", p, v) / torch.where(total > 0, total, 1.0)
    return o.flatten(1, 2), (torch.log(total) + top).squeeze(-1).flatten(1)


def run(state):
    s, case = state, state["case"]
    if own:
        import sparse_attention_indexer_exact_gb300 as gvr
        if case["op"] == "tables":
            slots, counts = gvr.cache_tables(s["cached"], s["lens"], s["free"], s["table"], s["new"], case["page_size"],
                                             case["cr"])
            return s["table"], slots, counts
        if case["op"] == "append":
            gvr.cache_append(s["k"], s["v"], s["cache"], s["slots"], v_scale=0.5)
            return gvr.cache_read(s["cache"], s["slots"], case["dim"], s["k"].dtype, v_scale=0.5)
        if case["op"] == "decode":
            return gvr.attend_decode(s["q"], s["cache"], s["table"], s["lens"], case["next_n"], case["cr"],
                                     s.get("indices"), want_lse=True)
        return gvr.attend_prefill(s["q"], s["cache"], s["table"], s["requests"], s["starts"], s["ends"], s["indices"],
                                  want_lse=True)
    if case["op"] == "tables":
        return _plain_tables(s)
    if case["op"] == "append":
        return _plain_append(s)
    o, lse = _attend(s, torch.float32)
    return o.to(s["q"].dtype), lse


# --------------------------------------------------------------------------- work and definition
def _mean_entries(case):
    """Expected entries that one row reads (lengths are uniform in [lo, hi])."""
    if case["op"] == "prefill":
        lengths = [max(1, case["longest"] * p // 16) for p in (1, 3, 8, 16)]
        total = sum(lengths)
        return sum(sum(min(case["k"], i * m / 64) for i in range(1, 65)) / 64 * m for m in lengths) / total
    lo, hi = case["lo"] / case["cr"], case["hi"] / case["cr"]
    n = (lo + hi) / 2
    if case["k"]:
        n = sum(min(case["k"], lo + (hi - lo) * (i + 0.5) / 64) for i in range(64)) / 64
    busy = (case["requests"] - 1) / case["requests"] if case["requests"] > 4 else 1.0
    return n * busy


def work(case):
    if case["op"] == "tables":
        new = case["requests"] * (case["new_lo"] + case["new_hi"]) / 2 / case["cr"]
        pages = new / case["page_size"]
        return {"bytes": 8 * case["requests"] + 8 * pages + 4 * _slot_room(case) + 12, "flops": 0}
    if case["op"] == "append":
        n, per = case["tokens"] - case["padded"], case["heads"] * case["dim"]
        # K and V in, codes and scales out and in again, K and V out (padding rows: zeros)
        return {"bytes": 4 * n * per + 2 * n * per * 9 / 8 + 4 * case["tokens"] * per + 8 * case["tokens"], "flops": 0}
    rows = case["rows"] if case["op"] == "prefill" else case["requests"] * case["next_n"]
    n, per = _mean_entries(case), case["kv_heads"] * case["dim"] * 9 / 8
    reads = rows * n * per
    if case["op"] == "prefill":  # rows of one request share its entries
        reads = min(reads, sum(max(1, case["longest"] * p // 16) for p in (1, 3, 8, 16)) * per)
    elif not case["k"]:  # so do the rows of one request that read everything
        reads = case["requests"] * n * per
    qo = rows * case["heads"] * (4 * case["dim"] + 4)
    return {"bytes": reads + qo + 4 * rows * case["k"], "flops": 4 * rows * n * case["heads"] * case["dim"]}


def _exact_quantised(x, factor):
    """Each value as the nearest code times scale, from distances in 64 bits (ties to the code whose last bit is 0)."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    b = x.double().unflatten(-1, (-1, 16))
    want = (b.abs().amax(-1, keepdim=True) / (6 * factor)).clamp(max=448.0)
    # e4m3: 8 steps an octave down to 2^-6, even steps of 2^-9 below
    step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
    scale = torch.round(want / step) * step * factor
    y = torch.where(scale > 0, b.abs() / torch.where(scale > 0, scale, 1.0), 0.0)
    best = torch.zeros_like(y)
    away = y.clone()
    for i in range(1, 8):
        off = (y - grid[i]).abs()
        better = (off < away) | ((off == away) & (i % 2 == 0))
        best, away = torch.where(better, grid[i], best), torch.where(better, off, away)
    return (best * b.sign() * scale).flatten(-2)


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        ok = (s["slots"] >= 0)[:, None, None]
        return _exact_quantised(s["k"], 1.0) * ok, _exact_quantised(s["v"], 0.5) * ok
    hk, d, ps = case["kv_heads"], case["dim"], case["page_size"]
    out, lse = [], []
    q = s["q"].double()
    signed = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda", dtype=torch.float64)
    for r in range(q.shape[0]):
        if case["op"] == "decode":
            m, j = int(s["lens"][r // case["next_n"]]), r % case["next_n"]
            req, n = r // case["next_n"], 0 if m < case["next_n"] else (m - case["next_n"] + j + 1) // case["cr"]
        else:
            req, n = int(s["requests"][r]), int(s["ends"][r]) - int(s["starts"][r])
        if case["k"]:
            e = s["indices"][r].long()
            e = e[e >= 0]
        else:
            e = torch.arange(n, device="cuda")
        if e.numel() == 0:
            out.append(torch.zeros(case["heads"], d, dtype=torch.float64, device="cuda"))
            lse.append(torch.full((case["heads"],), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        rows = s["cache"][s["table"][req, e // ps].long(), e % ps].transpose(0, 1)  # [hk, n, row]
        kv = []
        for i in (0, 1):
            codes = rows[..., i * (d // 2):(i + 1) * (d // 2)]
            x = torch.empty(*codes.shape[:-1], d, dtype=torch.float64, device="cuda")
            x[..., 0::2] = signed[(codes % 16).long()]
            x[..., 1::2] = signed[torch.div(codes, 16, rounding_mode="floor").long()]
            scales = rows[..., d + i * (d // 16):d + (i + 1) * (d // 16)].contiguous().view(torch.float8_e4m3fn)
            kv.append(x * scales.double().repeat_interleave(16, dim=-1))
        x = q[r].view(hk, -1, d) @ kv[0].transpose(1, 2) / math.sqrt(d)
        lse.append(torch.logsumexp(x, dim=-1).flatten())
        out.append((torch.softmax(x, dim=-1) @ kv[1]).flatten(0, 1))
    return torch.stack(out), torch.stack(lse)
