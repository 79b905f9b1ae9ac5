"""Attention of requests that share prefixes, on the GPU against sums in 64 bits over each request's own pages."""
from __future__ import annotations

import numpy as np
import pytest

import cachecheck

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = {torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -10}


@pytest.fixture(scope="module")
def gvr():
    import sparse_attention_indexer_exact_gb300 as mod
    mod.load_library()
    return mod


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def build(rng, groups, ps, kv_heads, dim, pool=512, k_scale=1.0, v_scale=1.0):
    """groups: (prefix, [entries behind it of each request]); entries below 0: an idle request without a table.  Full pages of a
    prefix are shared, the page that it ends in is each request's own copy.  Returns cache, table, entries, starts, prefixes."""
    k, v = (rng.standard_normal((pool, kv_heads, dim)).astype(np.float32) for _ in range(2))
    rows = cachecheck.pack(k, v, k_scale, v_scale)
    entries, starts, tables, free = [], [0], [], iter(())
    need = sum(p // ps + sum(-(-max(p + s, 0) // ps) - p // ps for s in own if s >= 0) for p, own in groups)
    order = rng.permutation(need + 3).astype(np.int32)
    free = iter(order)
    cache = rows[rng.integers(0, pool, (need + 3) * ps)].reshape(need + 3, ps, kv_heads, -1).copy()
    width = 1
    for p, own in groups:
        common = [next(free) for _ in range(p // ps)]
        first = None
        for s in own:
            if s < 0:
                entries.append(0)
                tables.append([])
                continue
            t = common + [next(free) for _ in range(-(-(p + s) // ps) - p // ps)]
            if p % ps and first is not None:
                cache[t[p // ps], :p % ps] = cache[first, :p % ps]
            if p % ps and first is None:
                first = t[p // ps]
            entries.append(p + s)
            tables.append(t)
            width = max(width, len(t))
        starts.append(starts[-1] + len(own))
    table = np.full((len(tables), width), -1, np.int32)
    for r, t in enumerate(tables):
        table[r, :len(t)] = t
    return cache, table, entries, np.array(starts, np.int32), np.array([p for p, _ in groups], np.int32)


def check(gvr, seed, groups, *, dim=128, dtype=torch.bfloat16, next_n=1, group=4, kv_heads=2, ps=16, cr=1, scale=None, cut_rows=0, strided=False,
          size=1.0, k_scale=1.0, v_scale=1.0, change=None, given=None, lens=None):
    rng = np.random.default_rng(seed)
    cache, table, entries, starts, prefixes = build(rng, groups, ps, kv_heads, dim, k_scale=k_scale, v_scale=v_scale)
    requests, heads = len(entries), group * kv_heads
    rows = requests * next_n - cut_rows
    # the last row of a request sees all of its entries
    kv = [n * cr + (n % cr) if n else 0 for n in entries] if lens is None else lens
    if change:
        change(cache, table, kv, starts, prefixes)
    q = torch.from_numpy((size * rng.standard_normal((rows, heads, dim))).astype(np.float32)).to(dtype)
    qd = q.cuda()
    if strided:
        qd = torch.full((rows, heads + 3, dim + 8), 9.0, dtype=dtype, device="cuda")[:, 1:heads + 1, :dim].copy_(q)
    s = 1 / np.sqrt(dim) if scale is None else scale
    if given is not None:
        starts, prefixes = (np.array(x, np.int32) for x in given)
    more = dict(scale=scale, want_lse=True, k_scale=k_scale, v_scale=v_scale)
    capacity = table.shape[1] * ps
    seen = cachecheck.row_entries(kv, next_n, cr, rows, capacity)
    ref = cachecheck.attend(q.double().numpy(), cache, table, seen, [r // next_n for r in range(rows)], None, s, k_scale, v_scale)
    v_max = np.nanmax(np.abs(cachecheck.unpack(cache, dim, k_scale, v_scale)[1]))
    tol, tol_lse = cachecheck.attend_tolerance(ref, EPS[dtype], v_max)
    # a table as narrow as it is, for which attend_decode's kernels may run, then one as wide as it takes for those of attend_shared
    wide = np.pad(table, ((0, 0), (0, -(-(1 << 25) // (requests * kv_heads * ps)))), constant_values=-1)
    for t in (table, wide):
        if t is wide and max(kv) // cr > capacity:
            continue  # it would show entries that the other one does not
        args = (qd, dev(cache), dev(t), dev(np.array(kv, np.int32)), next_n, cr, dev(starts), dev(prefixes))
        out, lse = gvr.attend_shared(*args, **more)
        assert out.dtype == dtype and out.shape == (rows, heads, dim) and lse.shape == (rows, heads)
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for got, want, most, name in ((o, ref[0], tol, "out"), (l, ref[1], tol_lse, "lse")):
            assert np.array_equal(np.isnan(got), np.isnan(want)), (name, np.argwhere(np.isnan(got) != np.isnan(want))[:5])
            with np.errstate(invalid="ignore"):
                bad = (np.abs(got - want) > most) & (got != want)
            assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], np.broadcast_to(most, got.shape)[bad][:5])
        again, lse2 = gvr.attend_shared(*args, **more)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(lse2.view(torch.int32), lse.view(torch.int32))  # the same bits
    return args, out, lse


@pytest.mark.parametrize("dim", [128, 64, 256])
def test_one_step(gvr, dim):
    """The smallest walk: one request, one step."""
    check(gvr, 1, [(0, [20])], dim=dim, group=1, kv_heads=1)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pair(gvr, dim):
    check(gvr, 2, [(200, [30, 7])], dim=dim)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("next_n,group,kv_heads", [(1, 8, 2), (2, 6, 1), (3, 1, 4)])
def test_groups(gvr, dim, dtype, next_n, group, kv_heads):
    """Prefixes that end in a page, at a page's end and within a step; requests of none, one and many entries behind them; a group of
    one and an empty one."""
    groups = [(300, [5, 100, 3, 260]), (64, [400, 3]), (777, [3]), (5, []), (1024, [33, -1, 700, 3, 4, 129, 128]), (0, [50, 3])]
    check(gvr, dim + next_n, groups, dim=dim, dtype=dtype, next_n=next_n, group=group, kv_heads=kv_heads, strided=True)


@pytest.mark.parametrize("members", [127, 128, 129, 255, 256, 257, 300])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_query_tiles(gvr, members, dim):
    """Queries of a group that fill a tile, both, and one more; one KV head, a row each."""
    check(gvr, members, [(500, [3] * members)], dim=dim, group=1, kv_heads=1)


@pytest.mark.parametrize("next_n,group", [(40, 8), (130, 1), (3, 100), (17, 16)])
def test_many_queries_a_request(gvr, next_n, group):
    """More queries a request than a tile, or two, hold; rows at the end that see less."""
    check(gvr, next_n, [(256, [150, 200 + next_n]), (100, [next_n, 300, 131])], group=group, kv_heads=1, dim=64, next_n=next_n, dtype=torch.float16)
    check(gvr, next_n, [(256, [150, 200 + next_n]), (100, [next_n, 300, 131])], group=group, kv_heads=1, dim=128, next_n=next_n, cut_rows=1)


def test_most_groups(gvr):
    """8192 groups, most of them empty, of requests whose many queries want the kernels of attend_shared all the same."""
    groups = [(70, [1, 2])] * 500 + [(1, [0])] * 24
    starts = list(range(0, 1002, 2)) + list(range(1001, 1025)) + [1024] * 7668
    check(gvr, 31, groups, dim=64, group=33, kv_heads=1, ps=2, given=(starts, [70] * 500 + [1] * 24 + [5] * 7668))


@pytest.mark.parametrize("next_n,group,left", [(300, 1, 10), (40, 8, 3), (1000, 1, 1), (130, 2, 129)])
@pytest.mark.parametrize("dim", [64, 256])
def test_a_last_request_of_fewer_rows(gvr, next_n, group, left, dim):
    """Of its query tiles only the first ones exist, alone and behind a prefix."""
    check(gvr, next_n, [(0, [next_n + 40])], group=group, kv_heads=2, dim=dim, next_n=next_n, cut_rows=next_n - left)
    check(gvr, next_n, [(100, [next_n + 40, next_n])], group=group, kv_heads=1, dim=dim, next_n=next_n, cut_rows=next_n - left)


@pytest.mark.parametrize("ps,cr", [(1, 1), (2, 4), (64, 4), (1024, 1), (4096, 2)])
def test_pages_and_ratios(gvr, ps, cr):
    check(gvr, ps, [(130, [5, 60, 300]), (1100, [1, 2])], ps=ps, cr=cr, next_n=2)


def test_no_groups_and_odd_ones(gvr):
    """Starts that fall, lie beyond the requests or below 0; prefixes of none, below 0 and beyond every length."""
    groups = [(300, [5, 100, 3, 260]), (300, [4, 9])]
    none = np.zeros(0, np.int32)
    check(gvr, 3, groups, given=(none, none))
    check(gvr, 3, groups, given=([0], none))
    check(gvr, 3, groups, given=([0, 4, 6], [-5, 0]))
    check(gvr, 3, groups, given=([0, 4, 6], [300, 2 ** 31 - 1]))
    check(gvr, 3, groups, given=([-7, 4, 2, 99], [300, 17, 200]))  # the second is empty, the third is requests 4 and 5
    check(gvr, 3, groups, given=([1, 3], [300]))  # requests 1 and 2; the others are in no group
    check(gvr, 3, groups, given=([6, 6, 9], [300, 300]))
    check(gvr, 3, groups, given=([0, 0, 0, 4, 4, 6, 6], [9, 9, 300, 9, 300, 9]))


def test_requests_shorter_than_the_prefix(gvr):
    """A request that does not see the whole prefix is attended by itself; the first of the group's may be one."""
    check(gvr, 4, [(300, [9, 20, 31, 42, 50])], lens=[299, 320, 0, 100, 350])
    check(gvr, 4, [(300, [9, 20, 31])], next_n=3, lens=[301, 303, 302])  # rows of 299, 300, 301: not all see it
    check(gvr, 4, [(300, [9, 20, 31])], lens=[100, 320, 2])  # one alone shares
    check(gvr, 4, [(300, [9, 20, 31])], lens=[1, 0, -4])


def test_no_entries_at_all(gvr):
    _, out, lse = check(gvr, 5, [(300, [9, 20])], lens=[0, 0])
    assert not out.any() and bool((lse == -np.inf).all())


def test_entries_on_no_page(gvr):
    def change(cache, table, kv, starts, prefixes):
        table[1, -1] = 10 ** 6
        table[:4, 3] = -1  # within the prefix, of all of its requests
        table[2, 25] = -2

    check(gvr, 6, [(300, [5, 200, 150, 260]), (0, [40, 5])], change=change)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nan_stays_with_those_who_see_it(gvr, dim):
    """NaN scales behind the last entry, and in entries that only later rows of a request see."""
    def change(cache, table, kv, starts, prefixes):
        ps = cache.shape[1]
        for r, n in enumerate(kv):
            if n % ps:
                cache[table[r, n // ps], n % ps:, :, dim:dim + dim // 8] = 127
        e = kv[1] - 2  # seen by the last two of four rows: V of one head's third block, and in the other request K
        cache[table[1, e // ps], e % ps, 0, dim + dim // 16 + 2] = 255
        e = kv[2] - 1
        cache[table[2, e // ps], e % ps, 1, dim + 1] = 127

    for prefix in (256, 0):
        check(gvr, 7, [(prefix, [40, 31, 77, 128]), (100, [29, 41])], dim=dim, next_n=4, change=change)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [70, 96, 130])
def test_nan_with_more_queries_than_two_tiles(gvr, dim, group):
    """Queries that fill tiles and those left over, in steps of either kind."""
    def change(cache, table, kv, starts, prefixes):
        ps = cache.shape[1]
        for r, back in ((0, 2), (1, 1)):
            e = kv[r] - back  # seen by the last rows of four
            cache[table[r, e // ps], e % ps, 0, dim + dim // 16 + 2] = 127

    check(gvr, 17, [(300, [140, 31])], dim=dim, next_n=4, group=group, kv_heads=1, change=change)


def test_nan_in_a_prefix_is_seen_by_all(gvr):
    def change(cache, table, kv, starts, prefixes):
        cache[table[0, 2], 5, 1, 128 + 8 + 3] = 127

    _, out, _ = check(gvr, 8, [(256, [40, 31]), (0, [60])], change=change)
    assert out.isnan().any(-1).any(-1).tolist() == [True, True, False]


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.5])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scales(gvr, scale, dtype):
    check(gvr, 9, [(300, [9, 200])], scale=scale, dtype=dtype, k_scale=0.5, v_scale=3.0)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_maxima_that_keep_growing(gvr, dim):
    """Keys that grow along the cache: bases are set again and again, and O is rescaled."""
    def change(cache, table, kv, starts, prefixes):
        for r in range(table.shape[0]):
            for b in range(-(-kv[r] // cache.shape[1])):
                cache[table[r, b], :, :, dim:dim + dim // 16] = min(0x20 + 2 * (b // 2), 0x70)

    check(gvr, 10, [(900, [9, 200, 150])], dim=dim, size=3.0, change=change)


def test_weights_far_apart(gvr):
    check(gvr, 11, [(900, [9, 200, 150])], size=30.0)
    check(gvr, 11, [(900, [9, 200, 150])], size=1e-20)


@pytest.mark.parametrize("dim,kv_heads,requests,prefix", [(128, 8, 33, 4000), (64, 1, 5, 40000), (256, 2, 9, 5000)])
def test_long_prefixes(gvr, dim, kv_heads, requests, prefix):
    """More steps than the device's SMs: units are cut within and between them."""
    rng = np.random.default_rng(12)
    check(gvr, 12, [(prefix, [int(x) for x in rng.integers(1, 90, requests)]), (prefix // 3, [4, 200])], dim=dim, kv_heads=kv_heads, group=2, ps=64)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("requests,next_n,cut_rows", [(2, 1, 0), (3, 3, 2)])
def test_few_queries_of_many_pieces(gvr, dim, requests, next_n, cut_rows):
    """Values whose pieces many threads join, beside short requests that have few."""
    check(gvr, 16, [(20000, [17] * requests), (0, [3])], dim=dim, kv_heads=1, group=2, next_n=next_n, cut_rows=cut_rows)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("next_n,group", [(1, 2), (3, 5), (1, 33)])
def test_few_and_many_entries_behind_a_prefix(gvr, dim, next_n, group):
    """On both sides of the 2048 that one CTA takes, with and without a prefix, which may end within a step of 32."""
    check(gvr, 18, [(0, [2047 + next_n]), (0, [2048]), (0, [2049]), (100, [1948 + next_n, 2041, 2049, 2148, 2149, 5, 31, 33, 1])], dim=dim,
          kv_heads=1, group=group, next_n=next_n)
    check(gvr, 19, [(0, [300, 2500, 31, 4000])], dim=dim, kv_heads=2, group=group, next_n=next_n, ps=8)


def test_many_requests(gvr):
    """1500 requests in 300 groups: more sets than the plan's CTA has threads."""
    rng = np.random.default_rng(13)
    groups = [(int(rng.integers(0, 60)), [int(x) for x in rng.integers(1, 30, 5)]) for _ in range(300)]
    check(gvr, 13, groups, dim=64, kv_heads=1, group=1)
    starts = np.arange(0, 1501, 5)
    assert len(starts) == 301


def test_same_as_attend_decode(gvr):
    """The plain call over the same arguments: both within their tolerances of the same sums, and alike to f16's roundings."""
    args, out, lse = check(gvr, 14, [(2000, [9, 200, 150, 31])], kv_heads=4, next_n=2, dtype=torch.float16)
    want, want_lse = gvr.attend_decode(*args[:6], want_lse=True)
    assert (out - want).abs().max() < 2e-3 and (lse - want_lse).abs().max() < 1e-4


def test_streams_graphs_and_given_outputs(gvr):
    args, out, lse = check(gvr, 15, [(500, [9, 200]), (100, [40, 41, 42])], kv_heads=2)
    o, l = torch.empty_like(out), torch.empty_like(lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gvr.attend_shared(*args, out=o, lse=l, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got[0] is o or got[0].data_ptr() == o.data_ptr()
    assert torch.equal(o, out) and torch.equal(l, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gvr.attend_shared(*args, out=o, lse=l)
    o.zero_()
    # the same graph over other lengths and prefixes
    for _ in range(2):
        graph.replay()
        assert torch.equal(o, out) and torch.equal(l, lse)
    args[7].zero_()
    graph.replay()
    want = gvr.attend_shared(*args)
    assert torch.equal(o, want[0])
    assert gvr.attend_shared(*args)[1] is None


def test_two_streams_at_once(gvr):
    """Calls that overlap: each has its own workspace, and tensor memory of its own SMs or its turn on them."""
    a, out_a, _ = check(gvr, 16, [(3000, [9, 200, 31])], kv_heads=2)
    b, out_b, _ = check(gvr, 17, [(2500, [90, 20])], kv_heads=4, dim=64, dtype=torch.float16)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for side, args in zip(sides, (a, b)):
            got.append(gvr.attend_shared(*args, stream=side)[0])
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, (out_a, out_b)[i % 2])
