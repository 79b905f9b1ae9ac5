"""Attention over the 4-bit cache where its numbers lie far apart, against 64-bit values of what the cache holds."""
from __future__ import annotations

import numpy as np
import pytest

import cachecheck as cc

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


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
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("n", [40, 1500, 207126])
@pytest.mark.parametrize("exponent", [-126, -118, 100, 116])
def test_factors_of_v_near_the_ends_of_fp32(gvr, n, exponent):
    """Equal weights of equal values: code * scale * v_scale, whatever the number of entries.  Every sum is exact (below
    2^24 steps), so the roundings left are the quotient's (2^-22 of the value in all) and the output's half step."""
    ps, vs = 4096, 2.0 ** exponent
    k = np.zeros((1, 1, 64), np.float32)
    v = np.tile(np.array([3.0, -6.0, 0.5, 1.5], np.float32), 16).reshape(1, 1, 64)
    cache = np.broadcast_to(cc.pack(k, v), (ps, 1, 80))[None].copy()
    table = np.zeros((1, -(-n // ps)), np.int64)
    q = torch.ones(1, 3, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = gvr.attend_decode(q, dev(cache, torch.uint8), dev(table), dev([n]), 1, 1, v_scale=vs, want_lse=True)
    want = v.reshape(-1).astype(np.float64) * vs
    assert np.abs(host(out) - want).max() <= 0  # each of them a bf16 number: half a step and 2^-22 lead back to it
    assert np.abs(host(lse) - np.log(n)).max() <= 2.0 ** -20 * np.log(n)
