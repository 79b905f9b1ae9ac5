"""What each entry draws, and eviction, on the GPU against plain implementations."""
from __future__ import annotations

import numpy as np
import pytest

import cachecheck
import longcheck

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gvr():
    import sparse_attention_indexer_exact_gb300 as mod
    mod.load_library()
    return mod


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def host(x):
    return x.cpu().numpy()


def random_cache(rng, pages, ps, heads, dim):
    """Rows as cache_append writes them, of normal values."""
    k, v = (rng.standard_normal((pages, ps, heads, dim)).astype(np.float32) for _ in range(2))
    return cachecheck.pack(k, v)


def paged(rng, entries, ps, extra=0, width=0):
    """A table [requests, width] of pages in random order, and the page numbers that no request holds."""
    need = [-(-int(n) // ps) for n in entries]
    width = max(width, max(need + [1]))
    order = rng.permutation(sum(need) + extra).astype(np.int32)
    table, at = np.full((len(need), width), -1, np.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table, order[at:].copy()


# --------------------------------------------------------------------------------------- weights
def weights_case(gvr, seed, *, dim, dtype, next_n, group, kv_heads, ps, cr=1, lens, scale=None, missing=False, cut_rows=0, poison=True,
                 strided=False, extra_columns=0):
    rng = np.random.default_rng(seed)
    requests, heads = len(lens), group * kv_heads
    rows = requests * next_n - cut_rows
    entries = [max(int(x), 0) // cr for x in lens]
    table, _ = paged(rng, entries, ps, extra=2)
    pages = int(table.max()) + 3
    cache = random_cache(rng, pages, ps, kv_heads, dim)
    if poison:  # NaN scales behind the last entry of each request
        for r, n in enumerate(entries):
            if n % ps:
                cache[table[r, n // ps], n % ps:, :, dim:dim + dim // 8] = 127
    if missing:
        table[0, 0], table[-1, table.shape[1] // 2] = -1, pages + 7
    q = torch.from_numpy(rng.standard_normal((rows, heads, dim)).astype(np.float32)).to(dtype)
    q64 = q.double().numpy()
    s = 1 / np.sqrt(dim) if scale is None else scale
    seen = cachecheck.row_entries(lens, next_n, cr, rows, table.shape[1] * ps)
    lse = cachecheck.attend(q64, cache, table, seen, [r // next_n for r in range(rows)], None, s)[1].astype(np.float32)
    width = table.shape[1] * ps + extra_columns
    before = rng.exponential(size=(requests, width)).astype(np.float32)
    qd = q.cuda()
    if strided:  # heads and rows apart
        qd = torch.full((rows, heads + 3, dim + 8), 9.0, dtype=dtype, device="cuda")[:, 1:heads + 1, :dim].copy_(q)
    w = dev(before)
    args = (qd, dev(cache), dev(table), dev(np.array(lens, np.int32)), next_n, cr, dev(lse))
    got = gvr.attend_weights(*args, w, scale=scale)
    assert got is w
    want, tol = longcheck.weights(q64, cache, table, lens, next_n, cr, lse, s, before)
    g = host(got).astype(np.float64)
    bad = np.abs(g - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], g[bad][:5], want[bad][:5], tol[bad][:5])
    untouched = tol == 0
    assert np.array_equal(host(got)[untouched], before[untouched])
    again = gvr.attend_weights(*args, dev(before), scale=scale)
    assert torch.equal(again, got)  # the same bits
    return args, before, got


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("next_n,group,kv_heads", [(1, 8, 2), (1, 1, 1), (2, 6, 4), (5, 3, 1)])
def test_weights(gvr, dim, dtype, next_n, group, kv_heads):
    lens = [0, 1, next_n, next_n - 1, 31, 32, 33, 64 + next_n, 700, -3, 257]
    weights_case(gvr, dim + next_n, dim=dim, dtype=dtype, next_n=next_n, group=group, kv_heads=kv_heads, ps=16, lens=lens, strided=next_n > 1)


@pytest.mark.parametrize("ps,cr", [(1, 1), (2, 4), (64, 4), (4096, 1)])
def test_weights_pages_and_ratios(gvr, ps, cr):
    weights_case(gvr, ps, dim=64, dtype=torch.bfloat16, next_n=3, group=4, kv_heads=3, ps=ps, cr=cr, lens=[5 * cr, 129 * cr + 3, 2, 400 * cr + 1], cut_rows=1,
                 extra_columns=5)


def test_weights_of_entries_on_no_page(gvr):
    weights_case(gvr, 3, dim=128, dtype=torch.float16, next_n=1, group=2, kv_heads=2, ps=16, lens=[100, 40, 300, 300], missing=True)


@pytest.mark.parametrize("scale", [0.0, -0.07, 0.5])
def test_weights_scales(gvr, scale):
    weights_case(gvr, 4, dim=128, dtype=torch.bfloat16, next_n=2, group=4, kv_heads=2, ps=16, lens=[100, 333], scale=scale)


def test_weights_more_queries_than_shared_memory_holds(gvr):
    """64 rows of 16 heads under each KV head: 128 tiles of eight, 32 at a time."""
    weights_case(gvr, 5, dim=128, dtype=torch.bfloat16, next_n=64, group=16, kv_heads=1, ps=16, lens=[150, 64, 63])
    weights_case(gvr, 6, dim=256, dtype=torch.float16, next_n=3, group=8, kv_heads=20, ps=16, lens=[70, 33])


def test_weights_many_requests_and_long_ones(gvr):
    weights_case(gvr, 7, dim=64, dtype=torch.float16, next_n=1, group=1, kv_heads=1, ps=16, lens=[int(x) for x in np.random.default_rng(1).integers(0, 60, 900)])
    weights_case(gvr, 8, dim=64, dtype=torch.float16, next_n=1, group=2, kv_heads=1, ps=64, lens=[20011, 3, 9000], poison=False)


def test_weights_from_zeros_on_a_stream_and_in_a_graph(gvr):
    args, before, got = weights_case(gvr, 9, dim=128, dtype=torch.bfloat16, next_n=2, group=4, kv_heads=2, ps=16, lens=[100, 333, 20])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fresh = gvr.attend_weights(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    sums = host(got).astype(np.float64) - before
    assert np.allclose(host(fresh), sums, rtol=1e-5, atol=1e-6) and fresh.shape == got.shape
    w = dev(before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gvr.attend_weights(*args, w)
    w.copy_(dev(before))
    graph.replay()
    assert torch.equal(w, got)
    graph.replay()  # a second step adds the same again
    assert np.allclose(host(w), before + 2 * sums, rtol=1e-5, atol=1e-6)


# ------------------------------------------------------------------------------------------ evict
def evict_case(gvr, seed, *, dim=64, kv_heads=2, ps=16, cr=1, lens, keep, recent, w=None, free=None, max_released=None, missing=(), shift=0, width=0,
               extra_columns=0):
    rng = np.random.default_rng(seed)
    entries = [max(int(x), 0) // cr for x in lens]
    table, spare = paged(rng, entries, ps, extra=len(lens) * -(-keep // ps) + 2, width=width)
    pages = int(max(table.max(), spare.max())) + 1
    cache = rng.integers(0, 256, (pages, ps, kv_heads, cachecheck.ROW_BYTES[dim]), dtype=np.uint8)
    if free is not None:
        spare = spare[:free]
    for r, b in missing:
        table[r, b] = -1
    columns = table.shape[1] * ps + extra_columns
    if w is None:
        w = lambda shape: rng.exponential(size=shape)  # noqa: E731
    weights = np.asarray(w((len(lens), columns)), np.float32)
    max_released = table.size if max_released is None else max_released
    # weights that begin `shift` floats behind an aligned address
    base = torch.zeros(weights.size + shift, dtype=torch.float32, device="cuda")
    wd = base[shift:].view(weights.shape)
    wd.copy_(dev(weights))
    cd, td, ld, fd = dev(cache), dev(table), dev(np.array(lens, np.int32)), dev(spare)
    kept, new, released, counts = gvr.cache_evict(wd, cd, td, ld, fd, keep, recent, cr, max_released)
    want = longcheck.evict(weights, cache, table, lens, cr, spare, keep, recent, max_released)
    for name, a, b in zip(("counts", "kept", "new_lens", "released", "table"), (counts, kept, new, released, td), (want[6], want[3], want[4], want[5], want[2])):
        assert np.array_equal(host(a), b), (name, host(a), b)
    assert np.array_equal(host(wd).view(np.uint32), want[0].view(np.uint32))
    assert np.array_equal(host(cd), want[1])
    return want


@pytest.mark.parametrize("dim,kv_heads", [(64, 1), (64, 4), (128, 8), (256, 2), (128, 33)])
@pytest.mark.parametrize("ps", [1, 16, 64])
def test_evict(gvr, dim, kv_heads, ps):
    evict_case(gvr, dim + ps, dim=dim, kv_heads=kv_heads, ps=ps, lens=[0, 1, 99, 100, 101, 250, 700, -5, 164], keep=100, recent=30)


@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (64, 0), (64, 64), (65, 64), (63, 1), (300, 17)])
@pytest.mark.parametrize("cr", [1, 4])
def test_evict_budgets(gvr, keep, recent, cr):
    lens = [x * cr + x % cr for x in (keep, keep + 1, keep - 1, 2 * keep + 5, 1000, 16 * (keep // 16 + 1))]
    evict_case(gvr, keep, lens=lens, keep=keep, recent=recent, cr=cr)


def special(kind):
    def make(shape):
        rng = np.random.default_rng(7)
        w = rng.standard_normal(shape).astype(np.float32)
        if kind == "equal":
            w[:] = 0.25
        elif kind == "two":
            w = np.where(w > 0, 1.0, 2.0).astype(np.float32)
        elif kind == "zeros":
            w = np.where(w > 0, np.float32(0.0), np.float32(-0.0))
        elif kind == "far":
            pick = rng.integers(0, 8, shape)
            for i, x in enumerate((np.inf, -np.inf, 1e-45, -1e-45, 3e38, 0.0)):
                w[pick == i] = x
        elif kind == "nan":
            w[rng.random(shape) < 0.2] = np.nan
            w.view(np.uint32)[rng.random(shape) < 0.1] = 0xffc00001  # a NaN with its sign set
        elif kind == "rising":
            w[:] = np.arange(shape[1])
        elif kind == "falling":
            w[:] = -np.arange(shape[1])
        elif kind == "close":  # the same but for the last digit's bits
            w = (np.float32(1.0) + rng.integers(0, 700, shape).astype(np.float32) * np.float32(2.0 ** -23)).astype(np.float32)
        return w
    return make


@pytest.mark.parametrize("kind", ["equal", "two", "zeros", "far", "nan", "rising", "falling", "close"])
@pytest.mark.parametrize("requests", [1, 5])
def test_evict_special_weights(gvr, kind, requests):
    """One request: a cluster of CTAs; several short ones: a CTA each."""
    lens = [9003] if requests == 1 else [700, 513, 300, 511, 900]
    evict_case(gvr, 11, lens=lens, keep=300, recent=40, w=special(kind), shift=3 if requests == 5 else 0)


def test_evict_nothing_changes_before_the_budget(gvr):
    """Falling weights: the first `keep` entries stay, and the page that they end in is made anew all the same."""
    want = evict_case(gvr, 12, lens=[500, 480], keep=200, recent=0, w=special("falling"))
    assert want[6][0] == 2
    want = evict_case(gvr, 13, lens=[500, 480], keep=192, recent=0, w=special("falling"))
    assert want[6][0] == 0


@pytest.mark.parametrize("free", [0, 1, 6, 7, 13, 14, 20, 21])
def test_evict_without_enough_pages(gvr, free):
    """Seven pages a request: those are served, in order, that there are pages for."""
    want = evict_case(gvr, 14, lens=[300, 50, 300, 300], keep=100, recent=10, free=free, w=special("rising"))
    assert want[6][2] == 3 - free // 7


def test_evict_missing_pages_and_short_lists(gvr):
    evict_case(gvr, 15, lens=[300, 400, 500, 90], keep=100, recent=10, missing=[(1, 3)])
    evict_case(gvr, 16, lens=[300, 400, 500, 90], keep=100, recent=10, missing=[(1, 26)], width=30, max_released=5, extra_columns=9)
    evict_case(gvr, 17, lens=[300, 400], keep=100, recent=10, max_released=0)


def test_evict_lengths_beyond_the_table(gvr):
    rng = np.random.default_rng(18)
    cache = dev(rng.integers(0, 256, (40, 16, 1, 80), dtype=np.uint8))
    table = dev(np.arange(20, dtype=np.int32).reshape(2, 10))
    w = dev(rng.random((2, 160)).astype(np.float32))
    want = longcheck.evict(host(w), host(cache), host(table), [100000, 161], 1, np.arange(20, 40), 50, 20, 20)
    kept, new, released, counts = gvr.cache_evict(w, cache, table, dev(np.array([100000, 161], np.int32)), dev(np.arange(20, 40, dtype=np.int32)), 50, 20, 1, 20)
    for a, b in zip((w, cache, table, kept, new, released, counts), want):
        assert np.array_equal(host(a), b)


@pytest.mark.parametrize("n,keep,requests", [(131072, 20000, 2), (450000, 3001, 1), (30000, 29999, 3)])
def test_evict_long(gvr, n, keep, requests):
    """450000 entries: more keys than a cluster holds in shared memory."""
    rng = np.random.default_rng(19)
    lens = [n - 7 * r for r in range(requests)]
    table, spare = paged(rng, lens, 64, extra=requests * -(-keep // 64))
    pages = int(max(table.max(), spare.max())) + 1
    cache = torch.randint(0, 256, (pages, 64, 1, 80), dtype=torch.uint8, device="cuda")
    w = rng.exponential(size=(requests, table.shape[1] * 64)).astype(np.float32)
    w[rng.random(w.shape) < 0.3] = 0.5
    td, wd, before = dev(table), dev(w), cache.clone()
    kept, new, _, counts = gvr.cache_evict(wd, cache, td, dev(np.array(lens, np.int32)), dev(spare), keep, 100, 1, 0)
    after = host(td)
    for r in range(requests):
        if lens[r] <= keep:
            assert np.array_equal(host(kept)[r], np.pad(np.arange(lens[r]), (0, keep - lens[r]), constant_values=-1))
            assert np.array_equal(after[r], table[r]) and np.array_equal(host(wd)[r], w[r])
            continue
        older = np.arange(lens[r] - 100)
        heavy = np.lexsort((older, -w[r, older].astype(np.float64)))[:keep - 100]
        stay = np.concatenate((np.sort(heavy), np.arange(lens[r] - 100, lens[r])))
        assert np.array_equal(host(kept)[r], stay)
        at = np.arange(keep)
        assert torch.equal(cache[dev(after[r, at // 64]).long(), dev(at % 64)], before[dev(table[r, stay // 64]).long(), dev(stay % 64)])
        assert np.array_equal(host(wd)[r, :keep], w[r, stay]) and not host(wd)[r, keep:lens[r]].any()
    held = torch.from_numpy(table[table >= 0].astype(np.int64)).cuda()
    assert torch.equal(cache[held], before[held])  # no page that was held is written


def test_evict_many_requests(gvr):
    lens = [int(x) for x in np.random.default_rng(20).integers(0, 90, 1500)]
    evict_case(gvr, 21, lens=lens, keep=40, recent=7, kv_heads=1)


def test_evict_outputs_streams_and_graphs(gvr):
    """Given outputs are used; a captured call does the same on every replay of the same inputs."""
    rng = np.random.default_rng(22)
    lens = [300, 90, 411]
    table, spare = paged(rng, lens, 16, extra=30)
    cache = rng.integers(0, 256, (int(max(table.max(), spare.max())) + 1, 16, 2, 80), dtype=np.uint8)
    w = rng.exponential(size=(3, table.shape[1] * 16)).astype(np.float32)
    want = longcheck.evict(w, cache, table, lens, 1, spare, 100, 10, 60)
    cd, td, wd = dev(cache), dev(table), dev(w)
    ld, fd = dev(np.array(lens, np.int32)), dev(spare)
    outs = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((3, 100), (3,), (60,), (3,))]

    def check():
        for a, b in zip((wd, cd, td, *outs), want):
            assert np.array_equal(host(a), b)

    def again():
        for a, b in ((wd, w), (td, table), (cd, cache)):
            a.copy_(dev(b))
        for o in outs:
            o.fill_(77)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gvr.cache_evict(wd, cd, td, ld, fd, 100, 10, 1, 60, *outs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(a is b or a.data_ptr() == b.data_ptr() for a, b in zip(got, outs))
    check()
    again()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gvr.cache_evict(wd, cd, td, ld, fd, 100, 10, 1, 60, *outs)
    for _ in range(2):
        again()
        graph.replay()
        check()


def test_evict_writes_lengths_in_place(gvr):
    """new_lens may be kv_lens: many chunks a request, which all need its old length."""
    rng = np.random.default_rng(23)
    lens = [9000, 700, 5001, 12000, 4999]
    table, spare = paged(rng, lens, 16, extra=5 * 320)
    cache = rng.integers(0, 256, (int(max(table.max(), spare.max())) + 1, 16, 1, 80), dtype=np.uint8)
    w = rng.exponential(size=(5, table.shape[1] * 16)).astype(np.float32)
    want = longcheck.evict(w, cache, table, lens, 1, spare, 5000, 10, 0)
    cd, td, wd, ld = dev(cache), dev(table), dev(w), dev(np.array(lens, np.int32))
    kept, new, _, counts = gvr.cache_evict(wd, cd, td, ld, dev(spare), 5000, 10, new_lens=ld)
    assert new.data_ptr() == ld.data_ptr()
    for a, b in zip((wd, cd, td, kept, ld, counts), (*want[:5], want[6])):
        assert np.array_equal(host(a), b)


def test_evict_of_no_requests(gvr):
    cache = gvr.cache_alloc(4, 16, 2, 64)
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    kept, new, released, counts = gvr.cache_evict(torch.zeros(0, 64, device="cuda"), cache, empty.view(0, 4), empty, empty, 5, 2, 1, 3)
    assert kept.shape == (0, 5) and new.numel() == 0 and released.tolist() == [-1] * 3 and counts.tolist() == [0, 0, 0]


def test_attention_after_eviction(gvr):
    """The calls as a serving step makes them: attention and its weights, eviction, then attention over what is left."""
    rng = np.random.default_rng(23)
    lens, keep, heads, dim, ps = [500, 60, 333], 128, 8, 64, 16
    table, spare = paged(rng, lens, ps, extra=30)
    cache = random_cache(rng, int(max(table.max(), spare.max())) + 1, ps, 2, dim)
    q = torch.from_numpy(rng.standard_normal((3, heads, dim)).astype(np.float32)).to(torch.bfloat16)
    cd, td, ld = dev(cache), dev(table), dev(np.array(lens, np.int32))
    _, lse = gvr.attend_decode(q.cuda(), cd, td, ld, 1, 1, want_lse=True)
    w = gvr.attend_weights(q.cuda(), cd, td, ld, 1, 1, lse)
    assert np.allclose(host(w).sum(1), heads, rtol=1e-4)  # softmax weights of each head add up to 1
    drawn = host(w)
    kept, new, _, counts = gvr.cache_evict(w, cd, td, ld, dev(spare), keep, 20, 1)
    assert new.tolist() == [128, 60, 128] and counts[2] == 0
    out, lse = gvr.attend_decode(q.cuda(), cd, td, new, 1, 1, want_lse=True)
    listed = np.full((3, keep), -1, np.int64)
    for r in range(3):
        stay = longcheck.chosen(drawn[r], lens[r], keep, 20) if lens[r] > keep else list(range(lens[r]))
        listed[r, :len(stay)] = stay
    assert np.array_equal(host(kept), listed)
    ref = cachecheck.attend(q.double().numpy(), cache, table, lens, range(3), listed, 1 / np.sqrt(dim))
    tol, tol_lse = cachecheck.attend_tolerance(ref, 2.0 ** -7, np.abs(cachecheck.unpack(cache, dim)[1]).max())
    assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol).all() and (np.abs(host(lse) - ref[1]) <= tol_lse).all()


def test_a_run_of_all_three(gvr):
    """Requests behind a common prompt: attention and what it draws over some steps, eviction, and the prefix that is left of it."""
    rng = np.random.default_rng(24)
    prefix, lens, keep, recent, heads, kv_heads, dim, ps, next_n = 150, [260, 190, 333, 177], 160, 30, 8, 2, 64, 16, 2
    table, spare = paged(rng, lens, ps, extra=60)
    cache = random_cache(rng, int(max(table.max(), spare.max())) + 1, ps, kv_heads, dim)
    table[1:, :prefix // ps] = table[0, :prefix // ps]
    for r in (1, 2, 3):
        cache[table[r, prefix // ps], :prefix % ps] = cache[table[0, prefix // ps], :prefix % ps]
    cd, td, ld = dev(cache), dev(table), dev(np.array(lens, np.int32))
    starts, w = dev(np.array([0, 4], np.int32)), torch.zeros(4, table.shape[1] * ps, device="cuda")

    def step(given, entries, pages, common):
        q = torch.from_numpy(rng.standard_normal((4 * next_n, heads, dim)).astype(np.float32)).half()
        out, lse = gvr.attend_shared(q.cuda(), cd, td, given, next_n, 1, starts, dev(np.array([common], np.int32)), want_lse=True)
        before = host(w).copy()
        gvr.attend_weights(q.cuda(), cd, td, given, next_n, 1, lse, w)
        seen = cachecheck.row_entries(entries, next_n, 1, 4 * next_n, pages.shape[1] * ps)
        now = host(cd)
        ref = cachecheck.attend(q.double().numpy(), now, pages, seen, [r // next_n for r in range(4 * next_n)], None, 1 / np.sqrt(dim))
        tol, tol_lse = cachecheck.attend_tolerance(ref, 2.0 ** -10, np.abs(cachecheck.unpack(now, dim)[1]).max())
        assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol).all() and (np.abs(host(lse) - ref[1]) <= tol_lse).all()
        after, off = longcheck.weights(q.double().numpy(), now, pages, entries, next_n, 1, host(lse), 1 / np.sqrt(dim), before)
        assert (np.abs(host(w) - after) <= off).all()

    for _ in range(3):
        step(ld, lens, table, prefix)
    drawn, held = host(w).copy(), table[table >= 0]
    kept, new, _, counts = gvr.cache_evict(w, cd, td, ld, dev(spare), keep, recent)
    assert new.tolist() == [keep] * 4 and counts[2] == 0 and np.array_equal(host(cd)[held], cache[held])
    for r in range(4):
        assert host(kept)[r].tolist() == longcheck.chosen(drawn[r], lens[r], keep, recent)
    # entries that all requests kept in the same places
    same = (host(kept) == host(kept)[0]).all(0) & (host(kept)[0] < prefix)
    common = int(same.argmin())
    step(new, [keep] * 4, host(td), common)


@pytest.mark.parametrize("ps", [4, 64])
def test_pages_beyond_32_bits(gvr, ps):
    """A cache of 5 GB, of which the last pages are read and written."""
    rng = np.random.default_rng(25)
    heads, kv_heads, dim, lens, keep, recent = 4, 2, 128, [300, 210], 100, 20
    table, spare = paged(rng, lens, ps, extra=2 * -(-keep // ps))
    few = int(max(table.max(), spare.max())) + 1
    cache = random_cache(rng, few, ps, kv_heads, dim)
    table[1, :96 // ps] = table[0, :96 // ps]
    pages = 5 * 2 ** 30 // (ps * kv_heads * 144)
    first = pages - few
    assert first * ps * kv_heads * 144 > 2 ** 32
    big = gvr.cache_alloc(pages, ps, kv_heads, dim)
    big[first:] = dev(cache)
    far = np.where(table >= 0, table + first, table)
    td, ld = dev(far), dev(np.array(lens, np.int32))
    q = torch.from_numpy(rng.standard_normal((2, heads, dim)).astype(np.float32)).to(torch.bfloat16)
    groups = dev(np.array([0, 2], np.int32)), dev(np.array([64], np.int32))
    out, lse = gvr.attend_shared(q.cuda(), big, td, ld, 1, 1, *groups, want_lse=True)
    near = gvr.attend_shared(q.cuda(), dev(cache), dev(table), ld, 1, 1, *groups, want_lse=True)
    assert torch.equal(out, near[0]) and torch.equal(lse, near[1])
    w = gvr.attend_weights(q.cuda(), big, td, ld, 1, 1, lse)
    assert torch.equal(w, gvr.attend_weights(q.cuda(), dev(cache), dev(table), ld, 1, 1, lse))
    want = longcheck.evict(host(w), cache, table, lens, 1, spare, keep, recent, 200)
    kept, new, released, counts = gvr.cache_evict(w, big, td, ld, dev(spare + np.int32(first)), keep, recent, 1, 200)
    assert np.array_equal(host(kept), want[3]) and np.array_equal(host(big[first:]), want[1]) and np.array_equal(host(counts), want[6])
    assert np.array_equal(host(td), np.where(want[2] >= 0, want[2] + first, want[2]))
    assert np.array_equal(host(released), np.where(want[5] >= 0, np.array(want[5]) + first, want[5]))
