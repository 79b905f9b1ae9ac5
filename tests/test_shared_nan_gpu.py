"""NaNs in the cache reach those who see them and nobody else, where attend_shared's CTAs have many short units in a row."""
from __future__ import annotations

import numpy as np
import pytest

from test_shared_gpu import check, gvr, torch  # noqa: F401 - gvr is a fixture

pytestmark = pytest.mark.gpu


def nan_in_v(cache, page, at, head, dim, block):
    cache[page, at, head, dim + dim // 16 + block] = 127


@pytest.mark.parametrize("dim,group,requests,most", [(256, 33, 500, 60), (256, 33, 300, 150), (128, 65, 500, 100), (128, 65, 300, 300), (64, 129, 250, 100)])
def test_nan_in_short_requests_one_after_the_other(gvr, dim, group, requests, most):  # noqa: F811
    """Requests of one step, or a few, with too many queries for tails: every third has a NaN in its last entry, of one KV head."""
    rng = np.random.default_rng(dim + most)

    def change(cache, table, kv, starts, prefixes):
        for r in range(0, requests, 3):
            e = kv[r] - 1
            nan_in_v(cache, table[r, e // 16], e % 16, r // 3 % 2, dim, r % (dim // 16))

    _, out, _ = check(gvr, 41, [(0, [int(x) for x in rng.integers(1, most, requests)])], dim=dim, group=group, change=change)
    assert out.isnan().any(-1).any(-1).tolist() == [r % 3 == 0 for r in range(requests)]


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nan_in_short_prefixes_one_after_the_other(gvr, dim):  # noqa: F811
    """Prefixes that end within a step, each of eight requests, under eight KV heads."""
    def change(cache, table, kv, starts, prefixes):
        for g in range(0, 150, 3):
            nan_in_v(cache, table[8 * g, 5], 9, g // 3 % 8, dim, g % (dim // 16))

    _, out, _ = check(gvr, 42, [(96, [1, 5, 2, 9, 1, 30, 3, 4])] * 150, dim=dim, group=1, kv_heads=8, change=change)
    assert out.isnan().any(-1).any(-1).tolist() == [r // 8 % 3 == 0 for r in range(1200)]


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 64), (128, 40), (256, 64)])
def test_nan_in_a_prefix_with_idle_requests(gvr, dim, group):  # noqa: F811
    """Idle requests of so many queries that whole warps have none that is live, in groups whose prefix has a NaN; the groups after
    them have none, and all of their requests are live."""
    idle = {g: g % 3 for g in range(0, 200, 2)}
    groups = [(96, [-1 if idle.get(g) == i else 3 + i for i in range(4)]) for g in range(200)]

    def change(cache, table, kv, starts, prefixes):
        for g in idle:
            r = 4 * g + (g % 3 == 0)
            nan_in_v(cache, table[r, 5], 9, g // 2 % 2, dim, g % (dim // 16))

    _, out, _ = check(gvr, 43, groups, dim=dim, group=group, change=change)
    assert out.isnan().any(-1).any(-1).tolist() == [g in idle and idle[g] != i for g in range(200) for i in range(4)]
