"""The 4-bit cache's operators on the GPU against the plain 64-bit implementation of cachecheck."""
from __future__ import annotations

import math

import numpy as np
import pytest

import cachecheck as cc

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def gvr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_indexer_exact_gb300 import _build
    _build.build_library()
    import sparse_attention_indexer_exact_gb300 as mod
    mod.load_library()
    torch.cuda.set_device(0)
    return mod


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).to(DEV)


def host(t):
    return t.detach().float().cpu().numpy() if t.dtype in (torch.bfloat16, torch.float16) else t.detach().cpu().numpy()


# ------------------------------------------------------------------------------------- tables
def check_tables(gvr, cached, lens, free, table, max_new, ps, cr, offset=0):
    want = cc.tables(cached, lens, free, table, max_new, ps, cr)
    t = dev(table)
    room = torch.full((max_new + offset + 3,), -77, dtype=torch.int32, device=DEV)
    slots, counts = gvr.cache_tables(dev(cached), dev(lens), dev(free), t, max_new, ps, cr, slots=room[offset:offset + max_new])
    assert np.array_equal(host(t), want[0])
    assert np.array_equal(host(slots), want[1])
    assert np.array_equal(host(counts), want[2])
    r = host(room)
    assert (r[:offset] == -77).all() and (r[offset + max_new:] == -77).all()


@pytest.mark.parametrize("requests,ps,cr", [(1, 1, 1), (1, 64, 4), (3, 16, 1), (31, 2, 3), (64, 64, 4), (513, 16, 1), (1025, 8, 2)])
@pytest.mark.parametrize("seed", [0, 1])
def test_tables(gvr, requests, ps, cr, seed):
    g = np.random.default_rng(100 * requests + seed)
    cached = g.integers(0, 300, requests)
    lens = cached + g.integers(0, [5, 400][seed], requests)
    lens[g.random(requests) < 0.2] = 0  # finished requests: no growth
    width = int(max(cached.max(), lens.max()) // cr // ps) + 2
    need = -(-(cached // cr) // ps)
    order = g.permutation(int(need.sum()) + requests * width)
    table = np.full((requests, width), -1)
    at = 0
    for q in range(requests):
        table[q, :need[q]] = order[at:at + need[q]]
        at += need[q]
    new = int(np.maximum(lens // cr - cached // cr, 0).sum())
    for extra, offset in ((0, 0), (37, 1), (-min(new, 5), 2)):
        check_tables(gvr, cached, lens, order[at:], table, new + extra, ps, cr, offset)


def test_tables_borders(gvr):
    """Empty pool, pool that ends inside a request, table too narrow, negative lengths, rollback, no
    requests, requests that already overflow their table, unused slots."""
    table = np.arange(12).reshape(3, 4) + 100
    for free in ([], [7], [7, 8, 9]):
        check_tables(gvr, [0, 5, 60], [40, 70, 64], free, table, 120, 16, 1)
    check_tables(gvr, [-5, 8, 30], [10, -1, 7], [1, 2, 3], table, 20, 16, 1)
    check_tables(gvr, [100, 100, 0], [140, 100, 1], [1, 2, 3], table, 50, 16, 1)  # 4 x 16 < 100
    check_tables(gvr, [0, 0, 0], [0, 0, 0], [1], table, 0, 16, 1)
    check_tables(gvr, [], [], [1], np.zeros((0, 4)), 9, 16, 1)
    t = np.full((2, 4), -1)
    t[0, 0] = 2 ** 31 - 1  # a page whose slots do not fit 31 bits: no slot
    check_tables(gvr, [3, 0], [5, 2], [1], t, 4, 16, 1)


@pytest.mark.parametrize("grow,new", [([0, 700, 1999], 9), ([3, 4, 1998], 2), ([1999], 1), ([], 0), ([0], 40)])
def test_tables_of_mostly_idle_requests(gvr, grow, new):
    """Runs of requests without new entries between the few that have some, within four neighbouring slots too."""
    g = np.random.default_rng(new)
    cached = g.integers(0, 60, 2000)
    lens = cached.copy()
    lens[grow] += new
    table, free = g.permutation(2000 * 13)[:2000 * 13].reshape(2000, 13), 26000 + g.permutation(30)
    for max_new in (0, 7, 20000):
        check_tables(gvr, cached, lens, free, table, max_new, 8, 1)


def test_tables_most_requests(gvr):
    n = gvr.MAX_CACHE_REQUESTS
    g = np.random.default_rng(5)
    cached, width = g.integers(0, 60, n), 9
    lens = cached + g.integers(0, 12, n)
    check_tables(gvr, cached, lens, np.arange(3 * n), np.full((n, width), 5), 6 * n, 8, 1)
    with pytest.raises(gvr.GvrError):
        check_tables(gvr, np.zeros(n + 1), np.zeros(n + 1), [1], np.zeros((n + 1, 1)), 1, 8, 1)


def test_tables_wide_stride_keeps_what_lies_between(gvr):
    whole = torch.full((5, 20), -9, dtype=torch.int32, device=DEV)
    t = whole[:, 3:9]
    gvr.cache_tables(dev([0] * 5), dev([33] * 5), dev(np.arange(50)), t, 200, 8, 1)
    want = np.full((5, 20), -9)
    want[:, 3:8] = np.arange(25).reshape(5, 5)
    assert np.array_equal(host(whole), want)


# ----------------------------------------------------------------------------- append and read
def check_append(gvr, k, v, cache, slots, ks=1.0, vs=1.0):
    """Appends and compares every byte of the cache; values back in both types."""
    before = host(cache).copy()
    flat = before.reshape(-1, *before.shape[2:]) if before.size else before
    rows = cc.pack(host(k), host(v), ks, vs)
    sl = host(slots)
    ps, n = cache.shape[1], cache.shape[0] * cache.shape[1]
    for t in range(len(sl)):
        if 0 <= sl[t] < n:
            flat[sl[t], :, :k.shape[2] * 9 // 8] = rows[t][:, :k.shape[2] * 9 // 8]  # the unused bytes stay
    gvr.cache_append(k, v, cache, slots, k_scale=ks, v_scale=vs)
    dim = k.shape[2]
    used = dim + dim // 8
    got = host(cache)
    gc, wc = cc.unpack(got, dim, ks, vs), cc.unpack(flat.reshape(got.shape), dim, ks, vs)
    for a, b in zip(gc, wc):
        assert np.array_equal(a, b, equal_nan=True)
    # bytes too, but for the sign of zeros (value-equal)
    same = got[..., dim:used] == flat.reshape(got.shape)[..., dim:used]
    assert same.all()
    assert np.array_equal(got[..., used:], flat.reshape(got.shape)[..., used:])
    for dt in (torch.bfloat16, torch.float16):
        rk, rv = gvr.cache_read(cache, slots, dim, dt, k_scale=ks, v_scale=vs)
        for r, w, f in ((rk, wc[0], ks), (rv, wc[1], vs)):
            w = w.reshape(-1, *w.shape[2:])
            want = np.stack([w[s] if 0 <= s < n else np.zeros(w.shape[1:]) for s in sl]) if len(sl) else np.zeros(r.shape)
            want = torch.as_tensor(want.astype(np.float32)).to(dt).float().numpy()
            assert np.array_equal(host(r), want, equal_nan=True)
    assert ps > 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,ps", [(1, 1, 16), (5, 3, 1), (67, 2, 16), (130, 8, 64)])
def test_append_and_read(gvr, dim, dtype, tokens, heads, ps):
    g = torch.Generator().manual_seed(dim + tokens)
    x = torch.randn(tokens, 2, heads, dim, generator=g) * torch.exp(2 * torch.randn(tokens, 2, heads, 1, generator=g))
    x[0, 0, 0, 16:32] = 0
    if tokens > 3:
        x[1, 0, 0, :16] = torch.tensor([6, .25, .75, -1.25, 1.75, 2.5, 3.5, -5, -.25, -.75, 1.25, 5, -6, 3, -2, 0.5])  # ties
        x[2, 1, 0, 3] = float("nan")
        x[3, 0, 0, 5] = float("inf")
        x[3, 1, 0, 5] = -float("inf")
        x[3, 1, 0, 16:32] *= 1e-6 / 50  # scales that underflow
    x = x.to(DT[dtype]).to(DEV)
    pages = tokens // ps + 2
    order = torch.randperm(pages * ps, generator=g)[:tokens].to(torch.int32)
    if tokens > 3:
        order[-1] = -1
        order[-2] = pages * ps
    cache = torch.randint(0, 120, (pages, ps, heads, cc.ROW_BYTES[dim]), generator=g, dtype=torch.uint8).to(DEV)
    for ks, vs in ((1.0, 1.0), (0.25, 8.0)):
        check_append(gvr, x[:, 0], x[:, 1], cache, order.to(DEV), ks, vs)


def test_append_strides_and_pages_apart(gvr):
    """K and V as slices of one projection, head-major K, pages with a gap between them."""
    g = torch.Generator().manual_seed(9)
    n, h, d, ps = 33, 4, 64, 8
    qkv = torch.randn(n, 5 * h * d, generator=g).to(torch.bfloat16).to(DEV)
    k, v = qkv[:, 3 * h * d:4 * h * d].view(n, h, d), qkv[:, 4 * h * d:].view(n, h, d)
    slots = torch.randperm(6 * ps, generator=g)[:n].to(torch.int32).to(DEV)
    whole = torch.full((6, 3, ps, h, 80), 7, dtype=torch.uint8, device=DEV)
    check_append(gvr, k, v, whole[:, 1], slots)
    assert (whole[:, 0] == 7).all() and (whole[:, 2] == 7).all()
    hm = torch.randn(h, n, d, generator=g).to(torch.bfloat16).to(DEV).transpose(0, 1)
    check_append(gvr, hm, v, whole[:, 2], slots)
    check_append(gvr, hm[:1].expand(n, h, d), v, whole[:, 2], slots)  # a token stride of 0


def test_append_nothing(gvr):
    cache = gvr.cache_alloc(2, 16, 2, 64, DEV)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    gvr.cache_append(none, none, cache, dev([]))
    k, v = gvr.cache_read(cache, dev([]), 64)
    assert k.shape == v.shape == (0, 2, 64) and int(cache.sum()) == 0


# ----------------------------------------------------------------------------------- attention
def random_cache(g, pages, ps, heads, dim, spread=1.0):
    kv = g.standard_normal((2, pages, ps, heads, dim)) * np.exp(spread * g.standard_normal((2, 1, 1, heads, dim)))
    return cc.pack(kv[0].astype(np.float32), kv[1].astype(np.float32))


def compare(out, lse, ref, cache, dim, vs=1.0):
    v = cc.unpack(host(cache), dim, 1.0, vs)[1]
    v_max = np.nanmax(np.abs(v)) if v.size else 0
    tol, tol_lse = cc.attend_tolerance(ref, torch.finfo(out.dtype).eps, v_max)
    o, l = host(out).astype(np.float64), host(lse).astype(np.float64)
    assert np.isfinite(o).all()
    worst = np.abs(o - ref[0]) / tol
    assert worst.max(initial=0) <= 1, f"out: {worst.max()} of the bound at {np.unravel_index(worst.argmax(), worst.shape)}"
    fin = np.isfinite(ref[1])
    assert np.array_equal(l[~fin], ref[1][~fin])
    worst = np.abs(l - ref[1])[fin] / tol_lse[fin]
    assert worst.max(initial=0) <= 1, f"lse: {worst.max()} of the bound"


def decode_case(gvr, seed, dim, dtype, kv_heads, group, ps, next_n, cr, lens, k, ks=1.0, vs=1.0, scale=None, qsize=1.0,
                spoil=True, spread=0.5, pages=None):
    g = np.random.default_rng(seed)
    lens = np.asarray(lens)
    requests, rows = len(lens), len(lens) * next_n
    width = max(1, -(-(int(lens.max()) // cr) // ps))
    if pages is None:
        pages = requests * width + 2
        cache = random_cache(g, pages, ps, kv_heads, dim, spread)
        table = g.permutation(pages)[:requests * width].reshape(requests, width)
    else:  # requests share them
        cache = random_cache(g, pages, ps, kv_heads, dim, spread)
        table = g.integers(0, pages, (requests, width))
    entries = cc.row_entries(lens, next_n, cr, rows, width * ps)
    if spoil and width > 1:
        table[0, 0], table[-1, -1] = -1, pages
        table[requests // 2, 1] = 2 ** 31 - 1
    idx = None
    if k:
        idx = np.full((rows, k), -1)
        for r in range(rows):
            n = entries[r]
            m = min(n, k)
            idx[r, :m] = g.permutation(n)[:m] if n > k else np.arange(m)
        if spoil and k >= 4:
            for r in range(0, rows, 2):
                idx[r, 0], idx[r, k // 2], idx[r, k - 1] = -2, entries[r], idx[r, 1]  # failed, beyond, twice
            if rows > 2:
                idx[1] = -1
    q = torch.as_tensor(g.standard_normal((rows, kv_heads * group, dim)) * qsize).to(DT[dtype]).to(DEV)
    out, lse = gvr.attend_decode(q, dev(cache, torch.uint8), dev(table), dev(lens), next_n, cr,
                                 None if idx is None else dev(idx), scale=scale, k_scale=ks, v_scale=vs, want_lse=True)
    s = 1 / math.sqrt(dim) if scale is None else scale
    ref = cc.attend(host(q), cache, table, entries, [r // next_n for r in range(rows)], idx, s, ks, vs)
    compare(out, lse, ref, torch.as_tensor(cache), dim, vs)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,kv_heads,dtype", [(1, 1, "bf16"), (4, 3, "f16"), (8, 2, "bf16"), (9, 1, "f16"), (40, 1, "bf16")])
@pytest.mark.parametrize("k", [1, 31, 33, 512])
def test_decode_selected(gvr, dim, group, kv_heads, dtype, k):
    decode_case(gvr, dim + group + k, dim, dtype, kv_heads, group, 16, 2, 1, [700, 40, 33, 1, 513], k)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,kv_heads,next_n,dtype", [(1, 2, 1, "bf16"), (3, 2, 2, "f16"), (8, 1, 1, "f16"), (5, 1, 4, "bf16"),
                                                         (16, 1, 3, "f16")])
@pytest.mark.parametrize("ps,cr", [(16, 1), (4, 3), (1, 1)])
def test_decode_whole(gvr, dim, group, kv_heads, next_n, dtype, ps, cr):
    decode_case(gvr, dim + group + ps, dim, dtype, kv_heads, group, ps, next_n, cr, [cr * 161, 0, cr * 31 + next_n, 5, cr * 64], 0)


@pytest.mark.parametrize("k", [0, 2048])
@pytest.mark.parametrize("requests,length", [(1, 5000), (9, 2500), (300, 40)])
def test_decode_splits(gvr, k, requests, length):
    """One item over a whole cluster, several clusters, more items than the device holds."""
    g = np.random.default_rng(requests)
    lens = g.integers(max(1, length // 2), length + 1, requests)
    decode_case(gvr, requests + k, 128, "bf16", 2, 4, 64, 1, 1, lens, k)


@pytest.mark.parametrize("qsize,scale,ks,vs", [(1e-4, None, 1.0, 1.0), (300.0, 1e-3, 1.0, 0.25), (3.0, -0.2, 4.0, 3.0),
                                               (1.0, 0.0, 1.0, 1.0), (8.0, None, 1.0, 1.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_decode_scales(gvr, qsize, scale, ks, vs, dtype):
    """Tiny and large queries, negative and zero factors, peaked and flat rows, cache factors."""
    decode_case(gvr, 77, 128, dtype, 2, 4, 16, 1, 1, [300, 90], 64, ks, vs, scale, qsize)
    decode_case(gvr, 78, 64, dtype, 2, 4, 16, 2, 1, [300, 90], 0, ks, vs, scale, qsize)


def test_decode_query_range_of_bf16(gvr):
    """bf16 queries far outside f16's range: 2^100 with a scale that brings the scores back."""
    decode_case(gvr, 5, 128, "bf16", 1, 4, 16, 1, 1, [200], 64, 1.0, 1.0, 2.0 ** -102, 2.0 ** 100)
    decode_case(gvr, 6, 128, "bf16", 1, 4, 16, 1, 1, [200], 64, 1.0, 1.0, 2.0 ** 88, 2.0 ** -90)


def test_decode_growing_scores(gvr):
    """Scores that climb along the row, so that the running maximum grows at every step."""
    g = np.random.default_rng(3)
    n, d = 640, 64
    base = g.standard_normal(d)
    k = base * np.linspace(0, 12, n)[:, None] + 0.3 * g.standard_normal((n, d))
    cache = cc.pack(k.astype(np.float32)[:, None], g.standard_normal((n, 1, d)).astype(np.float32)).reshape(40, 16, 1, 80)
    table = np.arange(40)[None]
    q = torch.as_tensor(np.stack([base, -base, 0.1 * base, 0 * base])[None]).to(torch.bfloat16).to(DEV)
    out, lse = gvr.attend_decode(q, dev(cache, torch.uint8), dev(table), dev([n]), 1, 1, want_lse=True)
    compare(out, lse, cc.attend(host(q), cache, table, [n], [0], None, 1 / 8), torch.as_tensor(cache), d)


def test_decode_idle_and_strided(gvr):
    """q as a slice of a projection, pages that lie apart, given outputs, requests without entries,
    a batch of only such requests."""
    g = np.random.default_rng(8)
    cache = random_cache(g, 12, 16, 2, 128)
    whole = torch.full((12, 2, 16, 2, 144), 255, dtype=torch.uint8, device=DEV)
    whole[:, 1] = dev(cache, torch.uint8)
    x = torch.as_tensor(g.standard_normal((3, 12, 128))).to(torch.float16).to(DEV)
    q = x[:, 2:10]
    lens = np.array([50, 0, 90])
    table = torch.full((3, 11), -3, dtype=torch.int32, device=DEV)
    table[:, 2:8] = dev(g.permutation(12)[:6])
    t = table[:, 2:8]
    out = torch.full((3, 8, 128), 7, dtype=torch.float16, device=DEV)
    lse = torch.zeros(3, 8, device=DEV)
    got = gvr.attend_decode(q, whole[:, 1], t, dev(lens), 1, 1, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    ref = cc.attend(host(q), cache, host(t), lens, [0, 1, 2], None, 1 / math.sqrt(128))
    compare(out, lse, ref, torch.as_tensor(cache), 128)
    assert (host(out)[1] == 0).all() and (host(lse)[1] == -np.inf).all()
    out, lse = gvr.attend_decode(q, whole[:, 1], t, dev([0, -4, 0]), 1, 1, want_lse=True)
    assert (host(out) == 0).all() and (host(lse) == -np.inf).all()
    out, _ = gvr.attend_decode(q[:0], whole[:, 1], t, dev(lens), 1, 1)
    assert out.shape == (0, 8, 128)
    empty = torch.empty(0, 16, 2, 144, dtype=torch.uint8, device=DEV)  # a cache without pages
    out, lse = gvr.attend_decode(q, empty, t, dev(lens), 1, 1, want_lse=True)
    assert (host(out) == 0).all() and (host(lse) == -np.inf).all()


def test_decode_masked_nan_stays_out(gvr):
    """NaN scales and codes at their largest in entries that a row does not see leave it untouched;
    in an entry that it sees they make that KV head NaN."""
    g = np.random.default_rng(4)
    cache = random_cache(g, 8, 16, 2, 64)
    lens, table = np.array([70]), np.arange(8)[None]
    clean = cache.copy()
    cache[70 // 16, 70 % 16:] = 0xff
    cache[70 // 16 + 1:] = 0x7f
    q = torch.as_tensor(g.standard_normal((1, 4, 64))).to(torch.bfloat16).to(DEV)
    idx = np.full((1, 100), -1)
    idx[0, :70] = g.permutation(70)
    idx[0, 70:80] = np.arange(70, 80)
    for i in (None, idx):
        out, lse = gvr.attend_decode(q, dev(cache, torch.uint8), dev(table), dev(lens), 1, 1, None if i is None else dev(i), want_lse=True)
        ref = cc.attend(host(q), clean, table, lens, [0], i, 1 / 8)
        compare(out, lse, ref, torch.as_tensor(clean), 64)
    cache[0, 3, 1, 64] = 0x7f  # K scale of entry 3, KV head 1
    out, lse = gvr.attend_decode(q, dev(cache, torch.uint8), dev(table), dev(lens), 1, 1, want_lse=True)
    assert np.isfinite(host(out)[0, :2]).all() and np.isnan(host(out)[0, 2:]).all() and np.isnan(host(lse)[0, 2:]).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("length,next_n,k,dtype", [(90, 1, 40, "bf16"), (90, 2, 0, "f16"), (2000, 2, 0, "bf16"), (2000, 1, 0, "f16")])
def test_decode_bad_query_stays_in_its_head(gvr, bad, length, next_n, k, dtype):
    """A query that is not finite spoils its own row and head, none that it shares a job with."""
    g = np.random.default_rng(length)
    cache, table, rows = random_cache(g, 130, 16, 2, 128), g.permutation(130)[:125][None], next_n
    lens = np.array([length])
    idx = g.permutation(length - next_n)[None, :k].repeat(rows, 0) if k else None
    q = torch.as_tensor(g.standard_normal((rows, 12, 128))).to(DT[dtype]).to(DEV)
    ref = cc.attend(host(q), cache, table, cc.row_entries(lens, next_n, 1, rows, 2000), [0] * rows, idx, 1 / math.sqrt(128))
    q[0, 4, 77] = bad
    out, lse = gvr.attend_decode(q, dev(cache, torch.uint8), dev(table), dev(lens), next_n, 1, None if idx is None else dev(idx),
                                 want_lse=True)
    assert not np.isfinite(host(out)[0, 4]).any() and not np.isfinite(host(lse)[0, 4])
    fine = np.ones((rows, 12), bool)
    fine[0, 4] = False
    out, lse, ref = out.reshape(-1, 128), lse.reshape(-1), [x.reshape(rows * 12, *x.shape[2:]) if x.ndim > 1 else x.repeat(12) for x in ref]
    keep = np.flatnonzero(fine.reshape(-1))
    compare(out[keep][:, None], lse[keep][:, None], [x[keep][:, None] if i < 4 else x[keep] for i, x in enumerate(ref)],
            torch.as_tensor(cache), 128)


@pytest.mark.parametrize("dim,dtype,group,kv_heads,k", [(64, "f16", 8, 2, 40), (128, "bf16", 8, 1, 512), (256, "bf16", 3, 2, 100)])
def test_prefill_selected(gvr, dim, dtype, group, kv_heads, k):
    g = np.random.default_rng(dim)
    lengths, ps = [37, 300, 64], 16
    start = np.array([0, 37, 337])
    req = np.concatenate([np.full(n, i) for i, n in enumerate(lengths)])[::7]
    pos = np.concatenate([np.arange(n) for n in lengths])[::7]
    starts, ends = start[req], start[req] + pos + 1
    req, starts, ends = (np.append(x, y) for x, y in ((req, [-1, 3, 1, 0]), (starts, [0, 0, 50, -9]), (ends, [9, 9, 50, 20])))
    width = 19
    cache = random_cache(g, 3 * width, ps, kv_heads, dim)
    table = g.permutation(3 * width).reshape(3, width)
    rows = len(req)
    n = [min(max(int(e) - max(int(s), 0), 0), width * ps) for s, e in zip(starts, ends)]
    idx = np.full((rows, k), -1)
    for r in range(rows):
        m = min(n[r], k)
        idx[r, :m] = g.permutation(n[r])[:m] if n[r] > k else np.arange(m)
    q = torch.as_tensor(g.standard_normal((rows, kv_heads * group, dim))).to(DT[dtype]).to(DEV)
    out, lse = gvr.attend_prefill(q, dev(cache, torch.uint8), dev(table), dev(req), dev(starts), dev(ends), dev(idx), want_lse=True)
    ref = cc.attend(host(q), cache, table, n, req, idx, 1 / math.sqrt(dim))
    compare(out, lse, ref, torch.as_tensor(cache), dim)


def test_same_result_every_time(gvr):
    """No atomics, a fixed order of sums: the same bits again, alone or beside other calls."""
    g = np.random.default_rng(1)
    cache, table = dev(random_cache(g, 64, 16, 2, 128), torch.uint8), dev(g.permutation(64).reshape(2, 32))
    q = torch.as_tensor(g.standard_normal((2, 8, 128))).to(torch.bfloat16).to(DEV)
    lens = dev([500, 300])
    first = [host(x) for x in gvr.attend_decode(q, cache, table, lens, 1, 1, want_lse=True)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            got.append(gvr.attend_decode(q, cache, table, lens, 1, 1, want_lse=True))
    torch.cuda.synchronize()
    for out, lse in got:
        assert np.array_equal(host(out), first[0]) and np.array_equal(host(lse), first[1])


# -------------------------------------------------- whole caches in equal shares, joined by a second kernel
@pytest.mark.parametrize("dim,dtype,kv_heads,group,next_n", [(64, "bf16", 1, 1, 1), (64, "f16", 4, 6, 2), (64, "bf16", 3, 33, 1),
                                                             (128, "bf16", 8, 4, 1), (128, "f16", 2, 8, 3), (128, "f16", 6, 12, 1),
                                                             (256, "bf16", 2, 8, 1), (256, "f16", 1, 5, 2)])
@pytest.mark.parametrize("lens", [[1537], [0, 0, 1602, 0], [1] * 40 + [1999], [1536, 33, 0, 32, 31, 1700, 2, 1569, 800, 64],
                                  [4000, 3999]])
def test_decode_shares(gvr, dim, dtype, kv_heads, group, next_n, lens):
    """One request over all shares, idle ones at the ends, many within one share, ends on and beside steps."""
    decode_case(gvr, dim + len(lens), dim, dtype, kv_heads, group, 16, next_n, 1, lens, 0, pages=80)


@pytest.mark.parametrize("requests", [150, 301, 1024, 1025])
def test_decode_shares_of_many_requests(gvr, requests):
    """Up to and beyond what is cut into equal shares; one long request among short ones."""
    g = np.random.default_rng(requests)
    lens = g.integers(0, 20, requests)
    lens[requests // 3] = 1600
    decode_case(gvr, requests, 64, "bf16", 1, 2, 32, 1, 1, lens, 0, pages=60)


@pytest.mark.parametrize("room", [16, 100_000, 1_000_000, 1 << 25])
@pytest.mark.parametrize("dim,kv_heads,group,next_n,lens", [(64, 4, 6, 2, [1700, 5, 3000]), (64, 3, 33, 1, [2100] * 3),
                                                            (128, 8, 4, 1, [4000]), (128, 2, 16, 1, [1999, 1, 0, 1800]),
                                                            (256, 2, 3, 2, [1600, 1700])])
def test_decode_shares_as_far_as_the_workspace_goes(gvr, monkeypatch, room, dim, kv_heads, group, next_n, lens):
    """A workspace without room for the shares (long rows in clusters), with just some and with enough: the same sums,
    and nothing written behind it."""
    from types import SimpleNamespace

    from sparse_attention_indexer_exact_gb300 import cache as mod
    buf = torch.full((room + 4096,), 171, dtype=torch.uint8, device=DEV)
    monkeypatch.setattr(mod, "_native", SimpleNamespace(attend_decode=lambda *a: None))
    monkeypatch.setattr(mod, "_WORKSPACE", room)
    monkeypatch.setattr(mod, "_workspace", lambda device: buf[:room])
    decode_case(gvr, dim + room % 7, dim, "bf16", kv_heads, group, 16, next_n, 1, lens, 0, pages=90)
    assert (buf[room:] == 171).all()


@pytest.mark.parametrize("length", [40, 2000])
def test_decode_shared_entries_of_partial_requests(gvr, length):
    """A last request of which only some rows are there, and lengths that some rows of a request share."""
    g = np.random.default_rng(length)
    ps, next_n, cr, width = 16, 4, 2, 130
    cache, table = random_cache(g, 2 * width, ps, 2, 64), g.permutation(2 * width).reshape(2, width)
    lens, rows = np.array([length, length + 3]), 6
    q = torch.as_tensor(g.standard_normal((rows, 6, 64))).to(torch.bfloat16).to(DEV)
    out, lse = gvr.attend_decode(q, dev(cache, torch.uint8), dev(table), dev(lens), next_n, cr, want_lse=True)
    ref = cc.attend(host(q), cache, table, cc.row_entries(lens, next_n, cr, rows, width * ps), [0, 0, 0, 0, 1, 1], None, 1 / 8)
    compare(out, lse, ref, torch.as_tensor(cache), 64)


@pytest.mark.parametrize("length,next_n,cr", [(70, 3, 1), (97, 4, 2), (2050, 3, 1), (4100, 4, 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_decode_nan_behind_a_row_that_others_see(gvr, length, next_n, cr, dim):
    """A NaN that the last row of a request sees and the rows before it do not."""
    g = np.random.default_rng(length)
    ps, width = 16, -(-length // 16)
    cache = random_cache(g, width, ps, 1, dim)
    lens, table = np.array([length]), np.arange(width)[None]
    entries = cc.row_entries(lens, next_n, cr, next_n, width * ps)
    q = torch.as_tensor(g.standard_normal((next_n, 3, dim))).to(torch.float16).to(DEV)
    bad = cache.copy()
    bad.reshape(width * ps, -1)[entries[-1] - 1:] = 0xff
    out, lse = gvr.attend_decode(q, dev(bad, torch.uint8), dev(table), dev(lens), next_n, cr, want_lse=True)
    ref = cc.attend(host(q), cache, table, entries, [0] * next_n, None, 1 / math.sqrt(dim))
    clean = [r for r in range(next_n) if entries[r] < entries[-1]]
    assert 0 < len(clean) < next_n
    compare(out[clean], lse[clean], [x[clean] for x in ref], torch.as_tensor(cache), dim)
    last = [r for r in range(next_n) if r not in clean]
    assert np.isnan(host(out)[last]).all() and np.isnan(host(lse)[last]).all()


def test_decode_shares_of_idle_requests_and_no_table(gvr):
    """A wide table of requests without entries, and a table without columns: zeros, whatever out held."""
    g = np.random.default_rng(2)
    cache = dev(random_cache(g, 4, 16, 2, 128), torch.uint8)
    q = torch.as_tensor(g.standard_normal((3, 4, 128))).to(torch.bfloat16).to(DEV)
    wide = torch.zeros(3, 200, dtype=torch.int32, device=DEV)
    for t, lens in ((wide, [0, 0, -5]), (wide[:, :0], [9, 4000, 0]), (torch.empty(3, 0, dtype=torch.int32, device=DEV), [1, 2, 3])):
        out, lse = torch.full_like(q, 7), torch.full((3, 4), 7.0, device=DEV)
        gvr.attend_decode(q, cache, t, dev(lens), 1, 1, out=out, lse=lse)
        assert (host(out) == 0).all() and (host(lse) == -np.inf).all()


@pytest.mark.parametrize("k", [2047, 2049, 8193, 9001])
def test_long_selections(gvr, k):
    """Selections long enough to be cut into shares, for decode rows and prefill rows, -1 pads among them."""
    g = np.random.default_rng(k)
    lens = np.array([9500, 700, 0, 8200])
    decode_case(gvr, k, 64, "bf16", 2, 3, 16, 1, 1, lens, k)
    width = 600
    cache, table = random_cache(g, 2 * width, 16, 2, 64), g.permutation(2 * width).reshape(2, width)
    req, starts, ends = np.array([1, 0, 5, 0]), np.array([3, 0, 0, 40]), np.array([9303, 9600, 70, 1000])
    n = [9300, 9600, 70, 960]
    idx = np.full((4, k), -1)
    for r in range(4):
        m = min(n[r], k)
        idx[r, :m] = g.permutation(n[r])[:m]
    q = torch.as_tensor(g.standard_normal((4, 6, 64))).to(torch.float16).to(DEV)
    out, lse = gvr.attend_prefill(q, dev(cache, torch.uint8), dev(table), dev(req), dev(starts), dev(ends), dev(idx), want_lse=True)
    compare(out, lse, cc.attend(host(q), cache, table, n, req, idx, 1 / 8), torch.as_tensor(cache), 64)


# ------------------------------------------------------------------------------- how calls are made
def long_case(g):
    cache, table = dev(random_cache(g, 300, 16, 2, 64), torch.uint8), dev(g.permutation(300).reshape(2, 150))
    q = torch.as_tensor(g.standard_normal((4, 8, 64))).to(torch.bfloat16).to(DEV)
    return q, cache, table, dev([2300, 1900]), 2, 1


def test_shares_at_once_and_in_two_graphs(gvr):
    """The same bits from calls on three streams at once, and from two captured graphs replayed beside each other."""
    args = [long_case(np.random.default_rng(i)) for i in range(3)]
    first = [[host(x) for x in gvr.attend_decode(*a, want_lse=True)] for a in args]
    streams, got, graphs = [torch.cuda.Stream() for _ in range(3)], [], []
    for i in range(2):
        graphs.append((torch.cuda.CUDAGraph(), []))
        with torch.cuda.graph(graphs[i][0]):
            for _ in range(3):
                graphs[i][1].append(gvr.attend_decode(*args[i], want_lse=True))
    torch.cuda.synchronize()
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            got.append((i % 3, gvr.attend_decode(*args[i % 3], want_lse=True)))
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i][0].replay()
    torch.cuda.synchronize()
    for i, graph in enumerate(graphs):
        got += [(i, x) for x in graph[1]]
    for i, (out, lse) in got:
        assert np.array_equal(host(out), first[i][0]) and np.array_equal(host(lse), first[i][1])


def every_call(gvr, **kw):
    """One call of each entry point; what they return, on the host."""
    g = np.random.default_rng(6)
    cache = gvr.cache_alloc(12, 16, 2, 64, DEV)
    kv = torch.as_tensor(g.standard_normal((2, 90, 2, 64))).to(torch.float16).to(DEV)
    q = torch.as_tensor(g.standard_normal((2, 4, 64))).to(torch.float16).to(DEV)
    table = torch.full((2, 6), -1, dtype=torch.int32, device=DEV)
    zero, lens, free, idx = dev([0, 0]), dev([50, 40]), dev(np.arange(12)[::-1].copy()), dev(g.integers(-1, 40, (2, 33)))
    torch.cuda.synchronize()
    slots, counts = gvr.cache_tables(zero, lens, free, table, 90, 16, **kw)
    gvr.cache_append(kv[0], kv[1], cache, slots, v_scale=0.5, **kw)
    got = [slots, counts, table, *gvr.cache_read(cache, slots, 64, torch.float16, v_scale=0.5, **kw)]
    got += gvr.attend_decode(q, cache, table, lens, 1, 1, idx, want_lse=True, **kw)
    got += gvr.attend_decode(q, cache, table, lens, 1, 1, scale=0.3, want_lse=True, **kw)
    got += gvr.attend_prefill(q, cache, table, dev([1, 0]), zero, lens, idx, want_lse=True, **kw)
    torch.cuda.synchronize()
    return [host(x) for x in got]


def test_streams_given(gvr):
    """stream= as a torch stream and as a raw handle: the same results as on the current one."""
    want, s = every_call(gvr), torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for a, b in zip(every_call(gvr, stream=stream), want):
            assert np.array_equal(a, b)


def test_default_stream_by_its_handle_and_streams_of_other_devices(gvr):
    """stream=0 is the default stream, not a new one; a stream of another device is refused."""
    from types import SimpleNamespace

    from sparse_attention_indexer_exact_gb300.cache import _current
    t = torch.zeros(1, device=DEV)
    with torch.cuda.stream(torch.cuda.Stream()):
        with _current(0, t):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
        for a, b in zip(every_call(gvr, stream=0), every_call(gvr)):
            assert np.array_equal(a, b)
    with pytest.raises(ValueError):
        _current(torch.cuda.Stream(), SimpleNamespace(device=torch.device("cuda", 1)))


def test_short_way_and_checked_way_agree(gvr, monkeypatch):
    """Ordinary calls take the native short way; the checked way behind it gives the same results."""
    from sparse_attention_indexer_exact_gb300 import cache as mod
    short, names, taken = mod._short(), ["cache_tables", "cache_append", "cache_read", "attend_decode", "attend_prefill"], []

    class Watched:
        pass

    def watch(name, through):
        def call(*args):
            got = getattr(short, name)(*args) if through else None
            taken.append((name, got is not None))
            return got
        return call

    results = []
    for through in (True, False):
        w = Watched()
        for name in names:
            setattr(w, name, watch(name, through))
        monkeypatch.setattr(mod, "_native", w)
        taken.clear()
        results.append(every_call(gvr))
        assert {n for n, _ in taken} == set(names) and all(t == through for _, t in taken)
    for a, b in zip(*results):
        assert np.array_equal(a, b)


FIRST_CALLS = """
import sys, torch
import sparse_attention_indexer_exact_gb300 as gvr
d = "cuda:0"
q, k = torch.randn(2, 8, 128, device=d).half(), torch.randn(20, 2, 128, device=d).half()
cache, table = torch.zeros(300, 16, 2, 144, dtype=torch.uint8, device=d), torch.arange(300, device=d).int().view(2, 150)
lens, cached, free = torch.tensor([2000, 40], device=d).int(), torch.tensor([1990, 30], device=d).int(), torch.arange(10, device=d).int()
idx = torch.arange(64, device=d).int().view(2, 32)
def step():
    slots, counts = gvr.cache_tables(cached, lens, free, table, 20, 16)
    gvr.cache_append(k, k, cache, slots)
    return [slots, counts, *gvr.cache_read(cache, slots, 128), *gvr.attend_decode(q, cache, table, lens, 1, 1, want_lse=True),
            *gvr.attend_decode(q, cache, table, lens, 1, 1, idx, want_lse=True)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = step()
graph.replay()
got = [x.clone() for x in captured]
assert got[1].tolist() == [20, 1, 0]
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("the same")
"""


def test_first_calls_of_a_process_are_captured(gvr):
    """Nothing of a first call (attributes, lookups, loading) is at odds with a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "the same" in run.stdout, run.stderr[-2000:]


@pytest.mark.parametrize("apart", [False, True])
def test_caches_beyond_32_bits(gvr, apart):
    """Entries more than 2^32 bytes from the cache's start; with pages apart, more than 2^31 16-byte units."""
    g = np.random.default_rng(9)
    ps, heads, dim, pages = 16, 2, 128, 1000
    stride = 36 * 10 ** 6 // 16 * 16 + 16 if apart else 16 * 2 * 144
    if not apart:
        pages = (1 << 32) // stride + 500
    memory = torch.empty(pages * stride, dtype=torch.uint8, device=DEV)
    cache = memory.as_strided((pages, ps, heads, 144), (stride, heads * 144, 144, 1))
    used = np.concatenate([[0], pages - 1 - g.permutation(400)[:9]])
    table, lens = g.permutation(used)[None], np.array([ps * 10 - 3])
    e = np.arange(lens[0])
    slots = table[0][e // ps] * ps + e % ps
    k, v = (torch.as_tensor(g.standard_normal((lens[0], heads, dim))).to(torch.bfloat16).to(DEV) for _ in range(2))
    gvr.cache_append(k, v, cache, dev(slots))
    rows = host(cache[dev(used, torch.int64)])
    small = np.argsort(used)[np.searchsorted(np.sort(used), table[0])][None]  # the same table over the used pages alone
    packed = cc.pack(host(k), host(v))
    assert np.array_equal(rows.reshape(-1, heads, 144)[small[0][e // ps] * ps + e % ps], packed)
    back = gvr.cache_read(cache, dev(slots), dim)
    want = cc.unpack(packed, dim)
    assert all(np.array_equal(host(b), w) for b, w in zip(back, want))
    q = torch.as_tensor(g.standard_normal((1, 8, dim))).to(torch.bfloat16).to(DEV)
    idx = g.permutation(lens[0])[:100][None]
    for i in (None, idx):
        out, lse = gvr.attend_decode(q, cache, dev(table), dev(lens), 1, 1, None if i is None else dev(i), want_lse=True)
        ref = cc.attend(host(q), rows, small, lens, [0], i, 1 / math.sqrt(dim))
        compare(out, lse, ref, torch.as_tensor(packed[:, None]), dim)


# ----------------------------------------------------------------------------- a step together
def step_inputs(g, gvr, lens, next_n, heads, kv_heads, dim, ps, stride):
    rows = len(lens) * next_n
    return dict(k=torch.as_tensor(g.standard_normal((rows, kv_heads, dim))).to(torch.bfloat16).to(DEV),
                v=torch.as_tensor(g.standard_normal((rows, kv_heads, dim))).to(torch.bfloat16).to(DEV),
                q=torch.as_tensor(g.standard_normal((rows, heads, dim))).to(torch.bfloat16).to(DEV),
                logits=torch.as_tensor(g.standard_normal((rows, stride))).to(torch.float32).to(DEV))


@pytest.mark.parametrize("captured", [False, True])
def test_decode_steps_together(gvr, captured):
    """Prompts written, then decode steps: tables, append, top-K, attention over the selection and over
    everything, eagerly or as one captured graph replayed while the lengths grow."""
    g = np.random.default_rng(12)
    heads, kv_heads, dim, ps, next_n, k, stride = 8, 2, 64, 16, 2, 512, 1024
    lens = np.array([600, 40, 701, 5])
    n, width, pages = len(lens), 60, 200
    cache = gvr.cache_alloc(pages, ps, kv_heads, dim, DEV)
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    free = dev(g.permutation(pages))
    # the prompts
    total = int(lens.sum())
    kv = torch.as_tensor(g.standard_normal((2, total, kv_heads, dim))).to(torch.bfloat16).to(DEV)
    slots, counts = gvr.cache_tables(dev([0] * n), dev(lens), free, table, total + 9, ps)
    gvr.cache_append(kv[0], kv[1], cache, slots)
    used = int(counts[1])
    assert counts.tolist() == [total, int((-(-lens // ps)).sum()), 0]
    # mirror on the host
    mirror = [cc.pack(host(kv[0][a:a + m]), host(kv[1][a:a + m])) for a, m in zip(np.cumsum(lens) - lens, lens)]
    cached, now = dev(lens), dev(lens + next_n)
    buf = step_inputs(g, gvr, lens, next_n, heads, kv_heads, dim, ps, stride)
    pool = torch.full((n,), -1, dtype=torch.int32, device=DEV)

    def step():
        slots, counts = gvr.cache_tables(cached, now, pool, table, n * next_n, ps)
        gvr.cache_append(buf["k"], buf["v"], cache, slots)
        idx, _ = gvr.topk_decode(buf["logits"], now, next_n, 1, k)
        sel = gvr.attend_decode(buf["q"], cache, table, now, next_n, 1, idx, want_lse=True)
        return slots, counts, idx, sel, gvr.attend_decode(buf["q"], cache, table, now, next_n, 1, want_lse=True)

    graph = None
    for i in range(4):
        new = step_inputs(g, gvr, lens, next_n, heads, kv_heads, dim, ps, stride)
        for name in buf:
            buf[name].copy_(new[name])
        cached.copy_(dev(lens))
        lens = lens + next_n
        now.copy_(dev(lens))
        pool.copy_(free[used:used + n])
        if captured and graph is None:
            warm = torch.cuda.Stream()
            warm.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(warm):
                gvr.topk_decode(buf["logits"], now, next_n, 1, k)
            torch.cuda.current_stream().wait_stream(warm)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = step()
        if captured:
            graph.replay()
        else:
            got = step()
        torch.cuda.synchronize()
        slots, counts, idx, sel, every = got
        used += int(counts[1])
        assert int(counts[0]) == n * next_n and int(counts[2]) == 0
        for q in range(n):
            rows = slice(q * next_n, (q + 1) * next_n)
            mirror[q] = np.concatenate([mirror[q], cc.pack(host(buf["k"][rows]), host(buf["v"][rows]))])
        # the plain form over the mirror: one request after the other as its own pages
        flat = np.concatenate(mirror)
        base = np.cumsum([len(m) for m in mirror]) - [len(m) for m in mirror]
        rows = n * next_n
        entries = cc.row_entries(lens, next_n, 1, rows, width * ps)
        for chosen, (out, lse) in ((host(idx), sel), (None, every)):
            parts = []
            for q in range(n):
                one = mirror[q][:, None]  # pages of one entry
                r = slice(q * next_n, (q + 1) * next_n)
                parts.append(cc.attend(host(buf["q"][r]), one, np.arange(len(one))[None], entries[r], [0] * next_n,
                                       None if chosen is None else chosen[r], 1 / 8))
            ref = [np.concatenate(x) for x in zip(*parts)]
            compare(out, lse, ref, torch.as_tensor(flat[:, None]), dim)
        assert base[0] == 0
