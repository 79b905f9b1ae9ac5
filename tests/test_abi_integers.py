"""Integers of the top-K bindings that do not fit the 32 bits that the library takes them in (no GPU needed: every refusal
comes before the library is called)."""
from __future__ import annotations

import pytest

A = 0x10000  # an aligned address that is never read


@pytest.fixture(scope="module")
def gvr():
    from sparse_attention_indexer_exact_gb300 import _build
    _build.build_library()
    import sparse_attention_indexer_exact_gb300 as mod
    mod.load_library()
    return mod


@pytest.mark.parametrize("beyond", [2 ** 31, 2 ** 32 + 1, -2 ** 32 + 1, 2 ** 70])
@pytest.mark.parametrize("which", ["next_n", "compress_ratio", "k"])
@pytest.mark.parametrize("rows", [0, 4])
def test_decode_calls(gvr, beyond, which, rows, monkeypatch):
    """next_n = 2^32 + 1 asks for one length for all rows, and cut to 1 it would read one for each.  Without rows no call
    gets as far as a launch."""
    class Never:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    if rows:
        monkeypatch.setattr(gvr, "load_library", Never)
    n = {"next_n": 1, "compress_ratio": 1, "k": 512, which: beyond}
    head = (A, 1024, rows, A, n["next_n"], n["compress_ratio"], n["k"])
    for call, rest in ((gvr.topk_decode_raw, (A, None, 0)), (gvr.topk_decode_ws_raw, (A, None, A, 1 << 24, 0)),
                       (gvr.topk_decode_hinted_raw, (A, 2048, A, None, 0)), (gvr.topk_decode_blockskip_raw, (A, 32, A, None, 0)),
                       (gvr.topk_decode_noalloc_raw, (A, None, 0))):
        with pytest.raises(ValueError, match="32 bits"):
            call(*head, *rest)


@pytest.mark.parametrize("k", [2 ** 31, 2 ** 32 + 512, -2 ** 40])
def test_prefill_calls(gvr, k):
    for call, rest in ((gvr.topk_prefill_raw, (A, 0)), (gvr.topk_prefill_ws_raw, (A, A, 1 << 24, 0))):
        with pytest.raises(ValueError, match="32 bits"):
            call(A, 1024, 0, A, A, k, *rest)
