"""Host-side checks of the 4-bit cache's C ABI and bindings (no GPU needed).

Every refusal of include/gvr_cache.h comes before any device work, so it is tested with addresses
that are never read; the kernels' index arithmetic (bad pages, offsets beyond 32 bits, the borders
of rows and windows) is compiled for the host and compared with plain Python."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import cachecheck

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gvr_cache.h")
INDEX = os.path.join(ROOT, "sparse_attention_indexer_exact_gb300", "csrc_cache")
A = 0x10000  # an aligned address that is never read
NULL, ALIGN, STRIDE, ARG = 1, 2, 3, 5


@pytest.fixture(scope="module")
def gvr():
    from sparse_attention_indexer_exact_gb300 import _build
    _build.build_library()
    import sparse_attention_indexer_exact_gb300 as mod
    mod.load_library()
    return mod


@pytest.fixture(scope="module")
def lib(gvr):
    return gvr.load_library()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(\w+)\s*\(", text, flags=re.M)))


def test_library_exports_what_the_header_declares(gvr, lib):
    assert set(declared()) == {"cache_row_bytes", "cache_tables", "cache_append", "cache_read", "attend_decode",
                               "attend_prefill", "gvr_cache_status_string"}
    for name in declared():
        assert hasattr(lib, name) and name in gvr.EXPORTED_SYMBOLS
    for name in ("cache_alloc", "cache_tables", "cache_append", "cache_read", "attend_decode", "attend_prefill"):
        assert name in gvr.__all__ and callable(getattr(gvr, name))


def test_status_strings(lib):
    for code in (0, NULL, ALIGN, STRIDE, ARG, 6):
        assert len(lib.gvr_cache_status_string(code)) > 1 and lib.gvr_cache_status_string(code) != b"unknown status"
    assert lib.gvr_cache_status_string(99) == b"unknown status"


def test_row_bytes(gvr, lib):
    for dim, want in cachecheck.ROW_BYTES.items():
        assert gvr.cache_row_bytes(dim) == want and dim + dim // 8 <= want and want % 16 == 0
    for dim in (0, -64, 32, 96, 512):
        with pytest.raises(gvr.GvrError):
            gvr.cache_row_bytes(dim)
    assert lib.cache_row_bytes(64, None) == NULL


def struct(**kw):
    from sparse_attention_indexer_exact_gb300.cache import _Cache
    f = dict(data=A, num_pages=10, page_stride=16 * 2 * 144, page_size=16, num_kv_heads=2, head_dim=128, reserved=0,
             k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return _Cache(*[f[n] for n, _ in _Cache._fields_])


BAD_CACHES = [(dict(data=None), NULL), (dict(data=A + 8), ALIGN), (dict(num_pages=-1), ARG),
              (dict(num_pages=1 << 27), ARG), (dict(page_stride=16 * 2 * 144 - 16), STRIDE),
              (dict(page_stride=16 * 2 * 144 + 8), STRIDE), (dict(page_stride=1 << 62), STRIDE),
              (dict(page_stride=1 << 33, num_pages=8), STRIDE), (dict(page_stride=144 << 25, num_pages=200), STRIDE),
              (dict(page_size=0), ARG), (dict(page_size=24), ARG), (dict(page_size=-16), ARG),
              (dict(page_size=8192, page_stride=8192 * 2 * 144), ARG), (dict(num_kv_heads=0), ARG), (dict(head_dim=96), ARG),
              (dict(reserved=1), ARG), (dict(k_scale=0.0), ARG), (dict(v_scale=-1.0), ARG),
              (dict(k_scale=float("nan")), ARG), (dict(v_scale=float("inf")), ARG)]


def caller(f, names, ok):
    def call(cache=None, **kw):
        args = dict(ok)
        args.update(kw)
        c = struct(**(cache or {}))
        return f(None if "null_cache" in args else ctypes.byref(c), *[args[n] for n in names])
    return call


def test_append_refusals(lib):
    names = ["k", "kt", "kh", "v", "vt", "vh", "dtype", "slots", "tokens", "stream"]
    call = caller(lib.cache_append, names, dict(k=A, kt=256, kh=128, v=A, vt=256, vh=128, dtype=0, slots=A, tokens=4,
                                                stream=None))
    for kw, want in BAD_CACHES:
        assert call(cache=kw) == want, kw
    assert call(null_cache=1) == NULL
    for kw, want in [(dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(k=A + 8), ALIGN),
                     (dict(v=A + 2), ALIGN), (dict(slots=A + 2), ALIGN), (dict(kt=252), STRIDE), (dict(kh=4), STRIDE),
                     (dict(vt=-256), STRIDE), (dict(vh=1 << 32), STRIDE), (dict(dtype=2), ARG), (dict(tokens=-1), ARG),
                     (dict(tokens=1 << 60), ARG)]:
        assert call(**kw) == want, kw
    assert call(tokens=0, k=None, v=None, slots=None) == 0


def test_read_refusals(lib):
    names = ["slots", "tokens", "dtype", "k", "v", "stream"]
    call = caller(lib.cache_read, names, dict(slots=A, tokens=4, dtype=1, k=A, v=A, stream=None))
    for kw, want in BAD_CACHES:
        assert call(cache=kw) == want, kw
    for kw, want in [(dict(slots=None), NULL), (dict(k=A + 8), ALIGN), (dict(v=A + 4), ALIGN), (dict(slots=A + 1), ALIGN),
                     (dict(dtype=-1), ARG), (dict(tokens=-3), ARG)]:
        assert call(**kw) == want, kw
    assert call(tokens=0, slots=None, k=None, v=None) == 0
    assert call(k=None, v=None) == 0


def test_tables_refusals(lib):
    names = ["cached", "lens", "requests", "cr", "ps", "free", "num_free", "table", "stride", "width", "slots", "num_slots",
             "counts", "stream"]
    ok = dict(cached=A, lens=A, requests=3, cr=1, ps=16, free=A, num_free=9, table=A, stride=8, width=8, slots=A,
              num_slots=40, counts=A, stream=None)

    def call(**kw):
        args = dict(ok)
        args.update(kw)
        return lib.cache_tables(*[args[n] for n in names])

    for kw, want in [(dict(cached=None), NULL), (dict(lens=None), NULL), (dict(free=None), NULL), (dict(table=None), NULL),
                     (dict(slots=None), NULL), (dict(counts=None), NULL), (dict(cached=A + 2), ALIGN),
                     (dict(slots=A + 1), ALIGN), (dict(counts=A + 2), ALIGN), (dict(table=A + 2), ALIGN),
                     (dict(requests=-1), ARG), (dict(requests=8193), ARG), (dict(cr=0), ARG), (dict(ps=48), ARG),
                     (dict(ps=0), ARG), (dict(num_free=-1), ARG), (dict(num_slots=-1), ARG), (dict(num_slots=1 << 31), ARG),
                     (dict(width=-1), ARG), (dict(width=1 << 28, stride=1 << 28), ARG), (dict(stride=7), STRIDE)]:
        assert call(**kw) == want, kw


ATTEND = dict(q=A, qr=512, qh=128, dtype=0, rows=4, heads=4, table=A, stride=8, width=8, indices=A, k=32, scale=0.1, out=A,
              lse=None, ws=A, ws_bytes=1 << 20, stream=None)
BAD_ATTEND = [(dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL), (dict(q=A + 8), ALIGN),
              (dict(out=A + 2), ALIGN), (dict(lse=A + 2), ALIGN), (dict(table=A + 2), ALIGN), (dict(indices=A + 2), ALIGN),
              (dict(ws=A + 8), ALIGN),
              (dict(qr=508), STRIDE), (dict(qh=-128), STRIDE), (dict(qh=1 << 33), STRIDE), (dict(stride=7), STRIDE),
              (dict(dtype=7), ARG), (dict(rows=-1), ARG), (dict(heads=3), ARG), (dict(heads=0), ARG), (dict(k=0), ARG),
              (dict(k=1 << 31), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
              (dict(width=-1), ARG), (dict(width=1 << 28, stride=1 << 28), ARG), (dict(rows=1 << 40), ARG)]


def test_attend_decode_refusals(lib):
    names = ["q", "qr", "qh", "dtype", "rows", "heads", "table", "stride", "width", "lens", "next_n", "cr", "indices", "k",
             "scale", "out", "lse", "ws", "ws_bytes", "stream"]
    call = caller(lib.attend_decode, names, dict(ATTEND, lens=A, next_n=2, cr=4))
    for kw, want in BAD_CACHES:
        assert call(cache=kw) == want, kw
    assert call(null_cache=1) == NULL
    for kw, want in BAD_ATTEND + [(dict(lens=None), NULL), (dict(lens=A + 1), ALIGN), (dict(next_n=0), ARG),
                                  (dict(next_n=5000), ARG), (dict(cr=0), ARG)]:
        assert call(**kw) == want, kw
    assert call(rows=0, q=None, out=None, table=None, lens=None, indices=None) == 0


def test_attend_prefill_refusals(lib):
    names = ["q", "qr", "qh", "dtype", "rows", "heads", "table", "stride", "width", "requests", "req", "starts", "ends",
             "indices", "k", "scale", "out", "lse", "ws", "ws_bytes", "stream"]
    call = caller(lib.attend_prefill, names, dict(ATTEND, requests=2, req=A, starts=A, ends=A))
    for kw, want in BAD_CACHES:
        assert call(cache=kw) == want, kw
    for kw, want in BAD_ATTEND + [(dict(req=None), NULL), (dict(starts=None), NULL), (dict(ends=None), NULL),
                                  (dict(indices=None), NULL), (dict(req=A + 2), ALIGN), (dict(ends=A + 2), ALIGN),
                                  (dict(requests=-1), ARG)]:
        assert call(**kw) == want, kw
    assert call(rows=0, q=None, out=None, table=None, req=None, starts=None, ends=None, indices=None) == 0


def test_attend_refuses_a_factor_beyond_fp32(lib):
    """scale and k_scale are finite, their product is not."""
    names = ["q", "qr", "qh", "dtype", "rows", "heads", "table", "stride", "width", "lens", "next_n", "cr", "indices", "k",
             "scale", "out", "lse", "ws", "ws_bytes", "stream"]
    call = caller(lib.attend_decode, names, dict(ATTEND, lens=A, next_n=2, cr=4))
    for scale in (3e38, -3e38):
        assert call(scale=scale) == ARG
        assert call(cache=dict(k_scale=10.0), scale=scale) == ARG
    assert call(cache=dict(k_scale=1e38), scale=10.0) == ARG


def test_bindings_refuse_host_tensors_and_wrong_shapes(gvr):
    torch = pytest.importorskip("torch")
    cache = torch.zeros(4, 16, 2, 144, dtype=torch.uint8)
    slots = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        gvr.cache_append(x, x, cache, slots)
    with pytest.raises(TypeError, match="CUDA"):
        gvr.cache_read(cache, slots, 128)
    with pytest.raises(TypeError, match="CUDA"):
        gvr.cache_tables(slots, slots, slots, torch.zeros(3, 4, dtype=torch.int32), 5, 16)
    with pytest.raises(TypeError, match="CUDA"):
        gvr.attend_decode(x, cache, torch.zeros(3, 4, dtype=torch.int32), slots, 1, 1)
    with pytest.raises(TypeError, match="CUDA"):
        gvr.attend_prefill(x, cache, torch.zeros(3, 4, dtype=torch.int32), slots, slots, slots, torch.zeros(3, 8, dtype=torch.int32))


HOST = r"""
#include <cstdio>
#include "gvr_cache_index.h"
using namespace gvrc;
int main() {
  long long a[8]; char f;
  while (std::scanf(" %c %lld %lld %lld %lld %lld %lld %lld %lld", &f, a, a+1, a+2, a+3, a+4, a+5, a+6, a+7) == 9) {
    long long r = 0;
    if (f == 'r') r = row_offset(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7]);
    if (f == 's') r = slot_offset(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
    if (f == 'o') r = slot_of(a[0], a[1], a[2]);
    if (f == 'd') r = decode_entries(a[0], a[1], a[2], a[3], a[4]);
    if (f == 'w') r = window_entries(a[0], a[1], a[2]);
    if (f == 'p') r = pages_of(a[0], a[1]);
    if (f == 'b') r = row_bytes(a[0]);
    if (f == 'u') r = row_unit(a[0], a[1], a[2], a[3], a[4], a[5]);
    if (f == 'f') r = units_fit(a[0], a[1], a[2]) ? unit_bytes(a[1], a[2]) : 0;
    std::printf("%lld\n", r);
  }
}
"""


def test_index_arithmetic_on_the_host(tmp_path):
    """Bad pages and slots have no address; good ones past 2^32 bytes have the right one."""
    src, exe = tmp_path / "index.cpp", tmp_path / "index"
    src.write_text(HOST)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", INDEX, str(src), "-o",
                    str(exe)], check=True, capture_output=True)
    top = 2 ** 31 - 1
    asked, want = [], []

    def ask(f, args, answer):
        asked.append(f + " " + " ".join(str(x) for x in (list(args) + [0] * 8)[:8]))
        want.append(answer)

    for shift in (0, 4, 12):
        ps = 1 << shift
        for pages in (0, 1, 7, top >> shift):
            for heads, row in ((1, 80), (8, 144), (3, 288)):
                stride = ps * heads * row + 32
                for page in (-2 ** 31, -2, -1, 0, 1, 6, pages - 1, pages, pages + 1, top):
                    if page > top:
                        continue
                    for entry in (0, 1, ps - 1, ps, 5 * ps + 3, top):
                        for head in (0, heads - 1):
                            ok = 0 <= page < pages
                            at = page * stride + ((entry % ps) * heads + head) * row
                            ask("r", (page, pages, entry, shift, stride, heads, head, row), at if ok else -1)
                for slot in (-2 ** 31, -1, 0, 1, ps, pages * ps - 1, pages * ps, top):
                    if slot > top:
                        continue
                    ok = 0 <= slot < pages * ps
                    at = slot // ps * stride + ((slot % ps) * heads + heads - 1) * row
                    ask("s", (slot, pages, shift, stride, heads, heads - 1, row), at if ok else -1)
        for page in (-5, -1, 0, 3, (top >> shift), top):
            for entry in (0, ps - 1, top):
                s = page * ps + entry % ps
                ask("o", (page, entry, shift), s if page >= 0 and s < top else -1)
        for n in (0, 1, ps, ps + 1, top):
            ask("p", (n, shift), -(-n // ps))
    # attention's 32-bit units: the same places as the 64-bit offsets, up to the largest cache that fits
    for shift, heads, row, gap in ((0, 1, 80, 0), (4, 8, 144, 0), (12, 3, 288, 0), (6, 2, 144, 16), (4, 8, 80, 48)):
        stride = (1 << shift) * heads * row + gap
        unit = row if stride % row == 0 else 16
        most = min((2 ** 32 - 1) // (stride // unit), top >> shift)
        for pages, fits in ((0, 1), (1, 1), (most, 1), ((2 ** 32 - 1) // (stride // unit) + 1, 0)):
            ask("f", (pages, stride, row), unit if fits else 0)
        for page in (0, 1, most - 1):
            for entry in (0, (1 << shift) - 1, 5 * (1 << shift), top):
                for head in (0, heads - 1):
                    at = page * stride + ((entry % (1 << shift)) * heads + head) * row
                    assert at % unit == 0 and at // unit < 2 ** 32
                    ask("u", (page, entry, shift, stride // unit, row // unit * heads, head * row // unit), at // unit)
    for kv in (-3, 0, 1, 2, 3, 4, 100, top):
        for next_n in (1, 2, 4096):
            for j in (0, next_n - 1):
                for ratio in (1, 4, top):
                    for cap in (0, 25, top):
                        ask("d", (kv, next_n, j, ratio, cap), 0 if kv < next_n else min((kv - next_n + j + 1) // ratio, cap))
    for start in (-2 ** 31, -1, 0, 5, top):
        for end in (-2 ** 31, -1, 0, 4, 5, 6, top):
            for cap in (0, 3, top):
                ask("w", (start, end, cap), min(max(end - max(start, 0), 0), cap))
    for dim, row in cachecheck.ROW_BYTES.items():
        ask("b", (dim,), row)
    r = subprocess.run([str(exe)], input="\n".join(asked) + "\n", capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-500:]
    got = [int(x) for x in r.stdout.split()]
    bad = [(a, g, w) for a, g, w in zip(asked, got, want) if g != w]
    assert len(got) == len(want) and not bad, bad[:5]


def test_plain_quantiser_pins():
    """The plain form itself, at values worked by hand: codes, ties, scales, NaN, saturation."""
    x = np.zeros((1, 64), np.float32)
    x[0, :8] = [6, 0.25, 0.75, -1.25, 1.75, 2.5, 3.5, -5]  # scale 1: every tie goes to the even code
    x[0, 16] = 448 * 6 * 4  # past the largest scale
    x[0, 17] = -448
    x[0, 32] = 2.0 ** -9 * 6 / 2 * 0.99  # a scale that rounds to 0
    x[0, 48] = np.nan
    code, sc = cachecheck.quantise(x, 1.0)
    v = cachecheck.dequantise(code, sc, 1.0)[0]
    assert v[:8].tolist() == [6, 0, 1, -1, 2, 2, 4, -4]
    assert v[16] == 448 * 6 and v[17] == -448 and v[32] == 0
    assert np.isnan(v[48:64]).all()
    assert cachecheck.E4M3[126] == 448 and cachecheck.E4M3[1] == 2.0 ** -9 and np.isnan(cachecheck.E4M3[127])
