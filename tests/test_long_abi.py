"""Host-side checks of include/gvr_long.h and its bindings (no GPU needed): every refusal comes before any device work, so
it is tested with addresses that are never read; how attend_shared's work is cut is compiled for the host."""
from __future__ import annotations

import ctypes
import glob
import os
import re
import subprocess

import pytest

from test_cache_abi import A, ALIGN, ARG, BAD_CACHES, NULL, STRIDE, caller, gvr, lib, struct  # noqa: F401
from test_cache_bindings import code

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_attention_indexer_exact_gb300")
HEADER = os.path.join(ROOT, "include", "gvr_long.h")
WORKSPACE = 7
NO_GPU = 6  # where the answer depends on the device's SMs
UNIT_WORK = 3  # of gvr_shares.h


def test_library_exports_what_the_header_declares(gvr, lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(\w+)\s*\(", text, flags=re.M))
    assert declared == {"attend_shared", "attend_shared_workspace", "attend_weights", "cache_evict", "cache_evict_workspace",
                        "gvr_long_status_string"}
    for name in declared:
        assert hasattr(lib, name) and name in gvr.EXPORTED_SYMBOLS
    for name in ("attend_shared", "attend_weights", "cache_evict", "MAX_LONG_REQUESTS"):
        assert name in gvr.__all__ and hasattr(gvr, name)
    assert f"GVR_LONG_MAX_REQUESTS {gvr.MAX_LONG_REQUESTS} " in open(HEADER).read()


def test_status_strings(lib):
    known = {code: lib.gvr_long_status_string(code) for code in (0, NULL, ALIGN, STRIDE, ARG, 6, WORKSPACE)}
    assert len(set(known.values())) == len(known) and all(len(s) > 1 and s != b"unknown status" for s in known.values())
    assert lib.gvr_long_status_string(99) == b"unknown status" and b"workspace" in known[WORKSPACE]


# ------------------------------------------------------------------------------------------------ C entries
ROWS = dict(q=A, qr=512, qh=128, dtype=0, rows=4, heads=4, table=A, stride=8, width=8, lens=A, next_n=2, cr=4, scale=0.1, stream=None)
BAD_ROWS = [(dict(q=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(q=A + 8), ALIGN), (dict(table=A + 2), ALIGN),
            (dict(lens=A + 1), ALIGN), (dict(qr=508), STRIDE), (dict(qh=-128), STRIDE), (dict(qh=1 << 33), STRIDE), (dict(stride=7), STRIDE),
            (dict(dtype=7), ARG), (dict(rows=-1), ARG), (dict(rows=2 * 8192 + 1), ARG), (dict(rows=2 ** 63 - 1), ARG), (dict(heads=3), ARG),
            (dict(heads=0), ARG), (dict(heads=(1 << 20) + 2), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
            (dict(scale=3e38), ARG), (dict(width=-1), ARG), (dict(width=1 << 28, stride=1 << 28), ARG),
            (dict(width=(1 << 27) - 4095, stride=1 << 28), ARG), (dict(next_n=0), ARG), (dict(next_n=4097), ARG), (dict(cr=0), ARG),
            (dict(next_n=4096, heads=2 * 129), ARG), (dict(next_n=1, heads=1 << 20, rows=129), None)]


def shared(lib, **ok):
    return caller(lib.attend_shared, ["q", "qr", "qh", "dtype", "rows", "heads", "table", "stride", "width", "lens", "next_n", "cr", "starts",
                                      "prefix", "groups", "scale", "out", "lse", "ws", "ws_bytes", "stream"],
                  dict(ROWS, starts=A, prefix=A, groups=2, out=A, lse=None, ws=A, ws_bytes=0, **ok))


def test_attend_shared_refusals(lib):
    call = shared(lib)
    for kw, want in BAD_CACHES:
        assert call(cache=kw) == want, kw
    assert call(null_cache=1) == NULL
    for kw, want in BAD_ROWS + [(dict(out=None), NULL), (dict(starts=None), NULL), (dict(prefix=None), NULL), (dict(out=A + 8), ALIGN),
                                (dict(lse=A + 2), ALIGN), (dict(starts=A + 2), ALIGN), (dict(prefix=A + 1), ALIGN), (dict(groups=-1), ARG),
                                (dict(groups=8193), ARG)]:
        assert call(**kw) == (ARG if want is None else want), kw  # (2^19 queries a row and KV head, 129 rows: beyond 2^26 in all)
    assert call(cache=dict(k_scale=1e38), scale=10.0) == ARG
    assert call(rows=0, q=None, out=None, table=None, lens=None, starts=None, prefix=None, ws=None) == 0
    # too much work to count in 32 bits: 8192 requests x 2 heads x 2^23 steps
    assert call(cache=dict(page_size=4096, page_stride=4096 * 288, num_pages=10), rows=8192, next_n=1, width=(1 << 18), stride=1 << 18) == ARG


def test_attend_shared_workspace_refusals(lib):
    size = ctypes.c_size_t(0)

    def call(kv_heads=2, dim=128, rows=4, heads=4, next_n=2, groups=1, at=ctypes.byref(size)):
        return lib.attend_shared_workspace(kv_heads, dim, rows, heads, next_n, groups, at)

    assert call(at=None) == NULL
    for kw in (dict(kv_heads=0), dict(kv_heads=65536, heads=65536), dict(dim=96), dict(rows=-1), dict(heads=0), dict(heads=3), dict(next_n=0),
               dict(next_n=4097), dict(groups=-1), dict(groups=8193), dict(rows=2 * 8192 + 1), dict(rows=2 ** 63 - 1), dict(heads=1 << 21),
               dict(next_n=4096, heads=2 * 129), dict(next_n=1, heads=1 << 20, rows=129)):
        assert call(**kw) == ARG, kw
    assert call() in (0, NO_GPU)


def test_attend_weights_refusals(lib):
    call = caller(lib.attend_weights, ["q", "qr", "qh", "dtype", "rows", "heads", "table", "stride", "width", "lens", "next_n", "cr", "lse",
                                       "scale", "weights", "w_stride", "stream"], dict(ROWS, lse=A, weights=A, w_stride=128))
    for kw, want in BAD_CACHES:
        assert call(cache=kw) == want, kw
    for kw, want in BAD_ROWS + [(dict(lse=None), NULL), (dict(weights=None), NULL), (dict(lse=A + 2), ALIGN), (dict(weights=A + 1), ALIGN),
                                (dict(w_stride=127), STRIDE), (dict(w_stride=1 << 31), STRIDE)]:
        if want is not None:
            assert call(**kw) == want, kw
    assert call(rows=0, q=None, table=None, lens=None, lse=None, weights=None) == 0


EVICT = dict(weights=A, w_stride=128, table=A, stride=8, width=8, lens=A, requests=3, cr=4, free=A, num_free=9, keep=20, recent=5, kept=A,
             new=A, released=A, most=30, counts=A, ws=A, ws_bytes=1 << 20, stream=None)


def test_cache_evict_refusals(lib):
    call = caller(lib.cache_evict, list(EVICT), EVICT)
    for kw, want in BAD_CACHES:
        assert call(cache=kw) == want, kw
    for kw, want in [(dict(weights=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(free=None), NULL),
                     (dict(kept=None), NULL), (dict(new=None), NULL), (dict(released=None), NULL), (dict(counts=None), NULL),
                     (dict(weights=A + 2), ALIGN), (dict(table=A + 1), ALIGN), (dict(lens=A + 2), ALIGN), (dict(free=A + 2), ALIGN),
                     (dict(kept=A + 2), ALIGN), (dict(new=A + 2), ALIGN), (dict(released=A + 2), ALIGN), (dict(counts=A + 2), ALIGN),
                     (dict(w_stride=127), STRIDE), (dict(w_stride=1 << 31), STRIDE), (dict(stride=7), STRIDE), (dict(stride=1 << 31), STRIDE),
                     (dict(requests=-1), ARG), (dict(requests=8193), ARG), (dict(cr=0), ARG), (dict(num_free=-1), ARG),
                     (dict(num_free=1 << 31), ARG), (dict(keep=0), ARG), (dict(keep=-3), ARG), (dict(recent=-1), ARG), (dict(recent=21), ARG),
                     (dict(most=-1), ARG), (dict(most=1 << 31), ARG), (dict(width=-1), ARG),
                     (dict(width=(1 << 27) - 4095, stride=1 << 28, w_stride=2 ** 31 - 1), ARG),
                     (dict(keep=2 ** 31 // 3), ARG), (dict(keep=2 ** 31 - 2 ** 16 + 1, requests=1, cr=1), ARG), (dict(keep=2 ** 29, recent=0, requests=1), ARG),
                     (dict(ws=None), WORKSPACE), (dict(ws=A + 8), WORKSPACE), (dict(ws_bytes=479), WORKSPACE)]:
        assert call(**kw) == want, kw


@pytest.mark.parametrize("requests,keep", [(0, 1), (1, 1), (3, 20), (8192, 1000), (1, 2 ** 31 - 2 ** 16)])
def test_cache_evict_workspace(lib, requests, keep):
    """Room for five words a request and two an entry."""
    size = ctypes.c_size_t(99)
    assert lib.cache_evict_workspace(requests, keep, ctypes.byref(size)) == 0
    assert size.value == -(-20 * requests // 16) * 16 + 2 * -(-4 * requests * keep // 16) * 16
    assert lib.cache_evict_workspace(requests, keep, None) == NULL
    for bad in ((-1, keep), (8193, keep), (requests, 0), (requests, -1), (1, 2 ** 31 - 2 ** 16 + 1), (8192, 2 ** 18)):
        assert lib.cache_evict_workspace(*bad, ctypes.byref(size)) == ARG


# ------------------------------------------------------------------------------------------------ sources
@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(PKG, "csrc_long", "*"))), ids=os.path.basename)
def test_nothing_is_read_as_read_only(path):
    """The kernels can be resident while the one before them still writes their inputs."""
    assert not re.findall(r"__ldg\w*|ld\.global\.nc|__restrict__", code(path))


def test_every_kernel_waits_for_the_one_before_it():
    kernels = 0
    for path in glob.glob(os.path.join(PKG, "csrc_long", "*.cu*")):
        for body in re.split(r"__global__", code(path))[1:]:
            kernels += 1
            assert re.search(r"\bbegin\(\);", body.split("\n}\n")[0])
    assert kernels == 7


SHARES = r"""
#include <cstdio>
#include <initializer_list>
#include "gvr_shares.h"
using namespace gvrc;
int main() {
  // lines: steps, both of each unit, then -1 and the CTAs.  Walks every share as the kernel does, and joins as it does.
  int steps[4096], both[4096], start[4097], n = 0, ctas;
  for (int units = 1; units < 7; ++units)  // of a set: its units one behind the other
    for (int full = 0; full <= units; ++full)
      for (int s : {1, 2, 5, 70})
        for (int u = 0, at = 0; u < units; ++u) {
          if (unit_start(u, full, s) != at) return 2;
          for (int end = at + unit_work(s, u < full); at < end; ++at)
            if (unit_at(at, full, s) != u) return 3;
          if (u + 1 == units && unit_start(units, full, s) != at) return 4;
        }
  while (std::scanf("%d", &steps[n]) == 1) {
    if (steps[n] >= 0) { if (std::scanf("%d", &both[n]) != 1) return 1; ++n; continue; }
    if (std::scanf("%d", &ctas) != 1) return 1;
    start[0] = 0;
    for (int u = 0; u < n; ++u) start[u + 1] = start[u] + unit_work(steps[u], both[u]);
    const int total = start[n];
    for (int c = 0, u = 0; c < ctas; ++c) {
      int at = share_start(c, ctas, total);
      const int last = share_start(c + 1, ctas, total);
      while (u > 0 && start[u] > at) --u;
      while (at < last) {
        while (start[u + 1] <= at) ++u;
        const int to = last < start[u + 1] ? last : start[u + 1];
        std::printf("walk %d %d %d %d\n", c, u, step_of(at, start[u], both[u], steps[u]), step_of(to, start[u], both[u], steps[u]));
        at = to;
      }
    }
    for (int u = 0; u < n; ++u)
      for (int c = share_of(start[u], ctas, total); c <= share_of(start[u + 1] - 1, ctas, total); ++c)
        std::printf("join %d %d %d %d\n", c, u, step_of(share_start(c, ctas, total), start[u], both[u], steps[u]),
                    step_of(share_start(c + 1, ctas, total), start[u], both[u], steps[u]));
    std::printf("end %d\n", total);
    n = 0;
  }
}
"""


def test_shares_are_joined_as_they_are_walked(tmp_path):
    """Every step of every unit lies in one share, and the join finds just the pieces that the walk leaves, at most two more than
    there are shares for the units of any one query."""
    import random
    src, exe = tmp_path / "shares.cpp", tmp_path / "shares"
    src.write_text(SHARES)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", os.path.join(PKG, "csrc_long"), str(src),
                    "-o", str(exe)], check=True, capture_output=True)
    rng = random.Random(5)
    cases = [([(1, 0)], 1), ([(1, 0)], 2), ([(1, 1)], 3), ([(10 ** 8, 1), (1, 0), (10 ** 8, 1)], 152), ([(1, 0)] * 1000, 152)]
    for _ in range(300):
        units = [(rng.choice([1, 2, 3, 7, 64, 513]), rng.randrange(2)) for _ in range(rng.randrange(1, 60))]
        total = sum(UNIT_WORK + (s << b) for s, b in units)
        cases.append((units, max(1, min(rng.choice([1, 3, 132, 152]), total // 2))))
    text = "\n".join(" ".join(f"{s} {b}" for s, b in units) + f" -1 {ctas}" for units, ctas in cases)
    r = subprocess.run([str(exe)], input=text, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-500:]
    at = iter(r.stdout.splitlines())
    for units, ctas in cases:
        walked, joined = {}, {}
        for line in at:
            kind, *x = line.split()
            if kind == "end":
                assert int(x[0]) == sum(UNIT_WORK + (s << b) for s, b in units)
                break
            c, u, lo, hi = map(int, x)
            assert 0 <= c < ctas
            if hi > lo:
                into = walked if kind == "walk" else joined
                assert (c, u) not in into
                into[c, u] = (lo, hi)
            if kind == "join":
                joined.setdefault(("count", u), 0)
                joined["count", u] += 1
        counts = [joined.pop(("count", u)) for u in range(len(units))]
        assert walked == joined
        if len(units) > 2:
            assert max(a + b + c for a, b, c in zip(counts, counts[1:], counts[2:])) <= ctas + 3
        for u, (steps, _) in enumerate(units):
            own = sorted(x for (c, w), x in walked.items() if w == u)
            assert own[0][0] == 0 and own[-1][1] == steps and all(a[1] == b[0] for a, b in zip(own, own[1:]))


# ------------------------------------------------------------------------------------------------ bindings
def calls(gvr, torch, **kw):
    i32, c, x = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 16, 2, 144, dtype=torch.uint8), torch.zeros(3, 2, 128).half()
    f32 = torch.zeros(3, 16)
    v = dict(next_n=1, cr=1, keep=4, recent=1, most=0)
    v.update(kw)
    return [lambda: gvr.attend_shared(x, c, i32[:, None], i32, v["next_n"], v["cr"], i32, i32[:2]),
            lambda: gvr.attend_weights(x, c, i32[:, None], i32, v["next_n"], v["cr"], f32[:, :2], f32),
            lambda: gvr.attend_weights(x, c, i32[:, None], i32, v["next_n"], v["cr"], f32[:, :2]),
            lambda: gvr.cache_evict(f32, c, i32[:, None], i32, i32, v["keep"], v["recent"], v["cr"], v["most"])]


def test_bindings_refuse_host_tensors(gvr):
    torch = pytest.importorskip("torch")
    for call in calls(gvr, torch):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_bindings_without_the_short_way_go_step_by_step(gvr, monkeypatch):
    import sys
    torch = pytest.importorskip("torch")
    from sparse_attention_indexer_exact_gb300 import cache
    monkeypatch.setattr(cache, "_native", None)
    monkeypatch.delattr(gvr, "_native", raising=False)
    monkeypatch.setitem(sys.modules, gvr.__name__ + "._native", None)
    first, *rest = calls(gvr, torch)
    with pytest.warns(RuntimeWarning, match="_native.so is missing"):
        with pytest.raises(TypeError, match="CUDA"):
            first()
    for call in rest:
        with pytest.raises(TypeError, match="CUDA"):
            call()


@pytest.mark.parametrize("beyond", [2 ** 31, 2 ** 32 + 1, -2 ** 31 - 1, 2 ** 70])
def test_integers_beyond_32_bits_are_refused(gvr, beyond):
    torch = pytest.importorskip("torch")
    for name, where in (("next_n", (0, 1, 2)), ("cr", (0, 1, 2, 3)), ("keep", (3,)), ("recent", (3,))):
        for i in where:
            with pytest.raises(ValueError, match={"cr": "compress_ratio"}.get(name, name)):
                calls(gvr, torch, **{name: beyond})[i]()


@pytest.mark.parametrize("keep,recent,most", [(0, 0, 0), (-1, 0, 0), (4, 5, 0), (4, -1, 0), (4, 1, -1)])
def test_evict_refuses_counts_that_make_no_sense(gvr, keep, recent, most):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="keep must be at least 1"):
        calls(gvr, torch, keep=keep, recent=recent, most=most)[3]()
