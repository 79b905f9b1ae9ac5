"""Which pages an eviction gave up: none of their numbers is lost unless the caller asks for fewer."""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np
import pytest

import longcheck
from test_long_gpu import dev, gvr, host, paged, torch  # noqa: F401 - gvr is a fixture

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["native", "checked"])
def way(request, monkeypatch):
    if request.param == "checked":
        from sparse_attention_indexer_exact_gb300 import cache
        monkeypatch.setattr(cache, "_native", SimpleNamespace(cache_evict=lambda *a: None))


def inputs(seed, lens, keep, ps=16, width=0):
    rng = np.random.default_rng(seed)
    table, spare = paged(rng, lens, ps, extra=len(lens) * -(-keep // ps), width=width)
    cache = rng.integers(0, 256, (int(max(table.max(), spare.max())) + 1, ps, 1, 80), dtype=np.uint8)
    return rng.exponential(size=(len(lens), table.shape[1] * ps)).astype(np.float32), cache, table, spare


def test_all_released_pages_are_listed(gvr, way):  # noqa: F811
    """Without max_released there is room for every page of the tables, which is the most that can be given up."""
    lens = [300, 90, 411, 100, 0]
    w, cache, table, spare = inputs(61, lens, 100, width=33)
    td = dev(table)
    want = longcheck.evict(w, cache, table, lens, 1, spare, 100, 10, table.size)
    got = gvr.cache_evict(dev(w), dev(cache), td, dev(np.array(lens, np.int32)), dev(spare), 100, 10)
    for a, b in zip((td, *got), (want[2], *want[3:])):
        assert np.array_equal(host(a), b)
    gone = host(got[2])[:int(got[3][1])]
    before, after = set(table[table >= 0].tolist()), set(host(td)[host(td) >= 0].tolist())
    assert set(gone.tolist()) == before - after and len(gone) == len(set(gone.tolist()))


def test_a_given_list_says_its_own_length(gvr, way):  # noqa: F811
    lens = [300, 411]
    for room in (0, 5, 26, 200):
        w, cache, table, spare = inputs(62, lens, 100)
        want = longcheck.evict(w, cache, table, lens, 1, spare, 100, 10, room)
        given = torch.full((room,), 77, dtype=torch.int32, device="cuda")
        got = gvr.cache_evict(dev(w), dev(cache), dev(table), dev(np.array(lens, np.int32)), dev(spare), 100, 10, released=given)
        assert got[2].data_ptr() == given.data_ptr() and np.array_equal(host(given), want[5]) and np.array_equal(host(got[3]), want[6])
    # asked for by number, as before
    w, cache, table, spare = inputs(62, lens, 100)
    got = gvr.cache_evict(dev(w), dev(cache), dev(table), dev(np.array(lens, np.int32)), dev(spare), 100, 10, 1, 0)
    assert got[2].numel() == 0 and host(got[3])[1] > 0
    with pytest.raises(ValueError, match="released"):
        gvr.cache_evict(dev(w), dev(cache), dev(table), dev(np.array(lens, np.int32)), dev(spare), 100, 10, 1, 4, released=given)


@pytest.mark.parametrize("lens", [[200, 40, 333], [40, 41], [5000], [150] * 700])
def test_long_lists_are_filled(gvr, way, lens):  # noqa: F811
    """Wide tables: far more room than pages, -1 behind the last one, whether requests are cut or not."""
    w, cache, table, spare = inputs(63, lens, 100, width=3000 if len(lens) < 10 else 300)
    want = longcheck.evict(w, cache, table, lens, 1, spare, 100, 10, table.size)
    got = gvr.cache_evict(dev(w), dev(cache), dev(table), dev(np.array(lens, np.int32)), dev(spare), 100, 10)
    for a, b in zip(got, want[3:]):
        assert np.array_equal(host(a), b)
    none = np.zeros(0, np.int32)
    kept, new, released, counts = gvr.cache_evict(dev(w), dev(cache), dev(table), dev(np.array(lens, np.int32)), dev(none), 100, 10)
    assert not (host(released) + 1).any() and host(counts)[:2].tolist() == [0, 0]
