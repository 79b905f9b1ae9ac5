"""attend_shared with lists of groups that are mostly empty, as a server pads them: what it asks of memory, and what it accepts."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from test_shared_gpu import build, dev, gvr, torch  # noqa: F401 - gvr is a fixture

pytestmark = pytest.mark.gpu


def space(gvr, kv_heads, dim, rows, heads, next_n, groups):  # noqa: F811
    lib, size = gvr.load_library(), ctypes.c_size_t(0)
    assert lib.attend_shared_workspace(kv_heads, dim, rows, heads, next_n, groups, ctypes.byref(size)) == 0
    return size.value


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("requests", [1, 2, 3, 64, 1001])
@pytest.mark.parametrize("next_n", [1, 2])
def test_groups_that_cannot_share_take_no_pieces(gvr, dim, requests, next_n):  # noqa: F811
    """At most half as many groups as requests share a prefix; what more are listed take their line in the plan, 48 bytes."""
    at_most = space(gvr, 8, dim, requests * next_n, 64, next_n, requests // 2)
    padded = space(gvr, 8, dim, requests * next_n, 64, next_n, 8192)
    assert 0 <= padded - at_most <= 48 * 8192


@pytest.mark.parametrize("requests", [1, 8])
def test_padded_groups_over_a_wide_table(gvr, requests):  # noqa: F811
    """8192 groups, one of which has requests, over tables of 4 million entries."""
    rng = np.random.default_rng(51)
    cache, table, entries, starts, prefixes = build(rng, [(300, [20 + 9 * r for r in range(requests)])], 16, 8, 128)
    big = np.zeros((requests, 4096, *cache.shape[2:]), np.uint8)  # pages of 4096 entries: one a request
    for r, n in enumerate(entries):
        for e in range(n):
            big[r, e] = cache[table[r, e // 16], e % 16]
    wide = np.full((requests, 1024), -1, np.int32)
    wide[:, 0] = np.arange(requests)
    q = torch.from_numpy(rng.standard_normal((requests, 16, 128)).astype(np.float32)).half().cuda()
    args = q, dev(big), dev(wide), dev(np.array(entries, np.int32)), 1, 1
    padded = np.concatenate((starts, np.full(8191, requests, np.int32)))
    out, lse = gvr.attend_shared(*args, dev(padded), dev(np.concatenate((prefixes, np.full(8191, 300, np.int32)))), want_lse=True)
    alone, alone_lse = gvr.attend_decode(*args, want_lse=True)
    assert (out - alone).abs().max() < 2e-3 and (lse - alone_lse).abs().max() < 1e-4
