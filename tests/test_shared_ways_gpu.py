"""attend_shared's cases through its own kernels, and through attend_decode's, whichever of them its rule would take."""
from __future__ import annotations

import ctypes
from types import SimpleNamespace

import numpy as np
import pytest

from test_long_gpu import test_a_run_of_all_three, test_pages_beyond_32_bits  # noqa: F401 - collected here too, with this file's gvr
from test_shared_gpu import *  # noqa: F401,F403 - its tests, with this file's gvr
from test_shared_gpu import build, check, dev
from test_shared_nan_gpu import *  # noqa: F401,F403

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BY_RULE, TOGETHER, APART = 0, 1, 2  # gvr_long_common.h


class Library:
    """The library, with attend_shared's way chosen; counts its calls."""

    def __init__(self, lib, way):
        self.lib, self.way, self.calls = lib, way, 0
        lib.attend_shared_way.argtypes = [ctypes.c_int32, *lib.attend_shared.argtypes]
        lib.attend_shared_way.restype = ctypes.c_int

    def attend_shared(self, *args):
        self.calls += 1
        return self.lib.attend_shared_way(self.way, *args)

    def __getattr__(self, name):
        return getattr(self.lib, name)


def take(gvr, monkeypatch, way):
    """Calls go step by step, through the Python binding's checks, to the library above."""
    from sparse_attention_indexer_exact_gb300 import cache
    native, lib = cache._short(), Library(gvr.load_library(), way)
    short = SimpleNamespace(**{name: getattr(native, name) for name in ("cache_tables", "cache_append", "cache_read", "attend_decode", "attend_prefill",
                                                                         "attend_weights", "cache_evict")}, attend_shared=lambda *a: None)
    monkeypatch.setattr(cache, "_native", short)
    monkeypatch.setattr(cache, "_library", lambda: lib)
    return lib


@pytest.fixture(params=[TOGETHER, APART], ids=["together", "apart"])
def gvr(request, monkeypatch):  # noqa: F811
    import sparse_attention_indexer_exact_gb300 as mod
    lib = take(mod, monkeypatch, request.param)
    yield mod
    assert lib.calls > 0


def test_most_requests_and_groups(gvr):
    """8192 of both, half of the groups empty: what the plan holds in shared memory at most."""
    rng = np.random.default_rng(44)
    groups = [(64, [int(x) for x in rng.integers(1, 30, 2)]) for _ in range(4096)]
    groups[7] = (40, [2100, 2060])
    starts = list(range(0, 8193, 2)) + [8192] * 4096
    check(gvr, 44, groups, dim=64, group=1, kv_heads=1, ps=2, given=(starts, [64] * 7 + [40] + [64] * 4088 + [5] * 4096))


def test_which_way_the_rule_takes(monkeypatch):
    """By the bits of the results: two requests in a narrow table apart, many behind a long prefix in a wide one together."""
    import sparse_attention_indexer_exact_gb300 as mod
    rng = np.random.default_rng(45)
    for requests, prefix, width, way in ((2, 500, 0, APART), (33, 4000, 4096, TOGETHER)):
        cache, table, entries, starts, prefixes = build(rng, [(prefix, [int(x) for x in rng.integers(1, 90, requests)])], 16, 8, 128)
        table = np.pad(table, ((0, 0), (0, max(0, width - table.shape[1]))), constant_values=-1)
        q = torch.from_numpy(rng.standard_normal((requests, 32, 128)).astype(np.float32)).half().cuda()
        args = (q, dev(cache), dev(table), dev(np.array(entries, np.int32)), 1, 1, dev(starts), dev(prefixes))
        outs = [mod.attend_shared(*args)[0]]
        for each in (BY_RULE, TOGETHER, APART):
            with monkeypatch.context() as m:
                take(mod, m, each)
                outs.append(mod.attend_shared(*args)[0])
        same = [torch.equal(outs[0], x) for x in outs[1:]]
        assert same == [True, way == TOGETHER, way == APART]
