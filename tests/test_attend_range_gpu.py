"""Attention over the 4-bit cache where its numbers lie far apart: one entry far above a long tail of others, and cache
factors near the ends of fp32's range, against 64-bit sums over what the cache holds.

The bound of an output element, from the documented roundings alone.  With weights w_e = exp(s_e - max s), S = sum w_e:
  relative  2^-11 of sum w|v| / S for the weights' 11-bit significands; 2^-17 for the exponentials, above and below the
            line (a score of at most 26 and its distance of at most 33 from the base, in log2 units, are rounded to 24
            bits: 2^-19.3 + 2^-19, and 2^-22 for the exponential itself); 2 n 2^-24 for the fp32 sums over n entries;
  absolute  half a step of the smallest f16 numbers, 2^-25, for each entry, where the largest weight of its walk is at
            least 2^7: n 2^-32 max|v| / S;
  and half a step of the output's type."""
from __future__ import annotations

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
    return t.detach().double().cpu().numpy()


def tail_cache(g, n, ps, gap, sinks, spread):
    """Pages in order of one KV head of 64: entries with scores near 0 against the query e_0, but for `sinks` (V = 0),
    whose score is near `gap`."""
    k, v = np.zeros((n, 64), np.float32), g.uniform(0.5, 2.0, (n, 64)).astype(np.float32)
    k[:, 0] = spread * g.standard_normal(n)
    k[sinks], v[sinks] = 0, 0
    k[sinks, 0] = gap
    pages = -(-n // ps)
    cache = np.zeros((pages * ps, 1, 80), np.uint8)
    cache[:n] = cc.pack(k[:, None], v[:, None])
    return cache.reshape(pages, ps, 1, 80)


def expected(cache, n, scale, v_scale):
    """(out, lse, sum w|v| / S, max|v| / S) of the query e_0 over the first n entries."""
    k, v = (x.reshape(-1, 64)[:n] for x in cc.unpack(cache, 64, 1.0, v_scale))
    s = scale * k[:, 0]
    w = np.exp(s - s.max())
    return w @ v / w.sum(), s.max() + np.log(w.sum()), w @ np.abs(v) / w.sum(), np.abs(v).max() / w.sum()


def check(out, lse, want, n, rows):
    """Every row and head of `out` and `lse` against the one expected row."""
    ref, ref_lse, spread, most = want
    eps = torch.finfo(out.dtype).eps
    tol = eps / 2 * np.abs(ref) + (1 + eps) * ((2.0 ** -11 + 2.0 ** -17 + 2 * n * 2.0 ** -24) * spread + n * 2.0 ** -32 * most)
    o, l = host(out).reshape(-1, 64), host(lse).reshape(-1)
    assert len(o) == rows
    worst = (np.abs(o - ref) / tol).max()
    assert worst <= 1, f"{worst} of the bound; largest relative difference {(np.abs(o - ref) / np.abs(ref)).max()}"
    assert np.abs(l - ref_lse).max() <= 2.0 ** -18 * (1 + abs(ref_lse)) + n * 2.0 ** -24


# scores of the entries above the tail, in nats: weights of the tail from 2^-17 to 2^-26 of the largest
GAPS = [12.0, 16.0, 17.5, 18.0]


def queries(rows, heads, dtype):
    q = torch.zeros(rows, heads, 64, dtype=DT[dtype], device=DEV)
    q[:, :, 0] = 1
    return q


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("spread", [0.0, 0.5])
@pytest.mark.parametrize("how", ["listed", "whole", "shares", "folded", "prefill"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tails_far_below_the_largest_weight(gvr, gap, spread, how, dtype):
    """A high entry in each step of 32, so that every walk has its base there, however a row is cut."""
    n = {"listed": 1500, "whole": 1500, "shares": 9000, "folded": 700, "prefill": 1500}[how]
    rows, next_n, ps, vs = 40, 3 if how == "folded" else 1, 16, 2.0 ** 20
    g = np.random.default_rng(int(10 * gap))
    cache = tail_cache(g, n, ps, gap, np.arange(0, n, 32), spread)
    table = np.arange(len(cache))[None].repeat(rows, 0)
    if how == "shares":
        rows, table = 2, table[:2]
    q, args = queries(rows, 6, dtype), (dev(cache, torch.uint8), dev(table))
    order = dev(np.stack([g.permutation(n) for _ in range(rows)]))
    if how == "prefill":
        out, lse = gvr.attend_prefill(q, *args, dev(np.arange(rows)), dev([0] * rows), dev([n] * rows), order, scale=1.0, v_scale=vs,
                                      want_lse=True)
    else:
        # all rows of a request but its last are one entry short of the next: the last one is compared
        out, lse = gvr.attend_decode(q, *args, dev([n] * rows), next_n, 1, order if how == "listed" else None, scale=1.0, v_scale=vs,
                                     want_lse=True)
    out, lse = out[next_n - 1::next_n], lse[next_n - 1::next_n]
    check(out, lse, expected(cache, n, 1.0, vs), n, rows // next_n * 6)


@pytest.mark.parametrize("gap", [15.0, 17.7])
@pytest.mark.parametrize("rows", [1, 1030])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_rows_behind_one_high_entry(gvr, gap, rows, dtype):
    """One entry above 131072 equal ones: cut into shares, or (many requests that share their pages) walked as they are."""
    n, ps, vs = 131073, 4096, 2.0 ** 10
    cache = tail_cache(np.random.default_rng(1), n, ps, gap, [0], 0.0)
    table = np.arange(len(cache))[None].repeat(rows, 0)
    out, lse = gvr.attend_decode(queries(rows, 2, dtype), dev(cache, torch.uint8), dev(table), dev([n] * rows), 1, 1, scale=1.0,
                                 v_scale=vs, want_lse=True)
    check(out, lse, expected(cache, n, 1.0, vs), n, rows * 2)


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
