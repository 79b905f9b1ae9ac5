"""Which attention calls take equal shares of their workspace: they write to it, and clusters do not."""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np
import pytest

from test_cache_gpu import DEV, decode_case, gvr  # noqa: F401 - gvr is a fixture

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
FILL = 171


@pytest.fixture
def workspace(monkeypatch):
    """The memory that calls are given; a call takes the checked way, which asks for it by _workspace."""
    from sparse_attention_indexer_exact_gb300 import cache as mod
    buf = torch.full((mod._WORKSPACE,), FILL, dtype=torch.uint8, device=DEV)
    monkeypatch.setattr(mod, "_native", SimpleNamespace(attend_decode=lambda *a: None))
    monkeypatch.setattr(mod, "_workspace", lambda device: buf[:mod._WORKSPACE])
    return buf


def written(buf) -> bool:
    return bool((buf != FILL).any())


@pytest.mark.parametrize("dim,dtype,kv_heads,group,next_n", [(64, "bf16", 1, 1, 1), (64, "f16", 4, 6, 2), (64, "bf16", 3, 33, 1),
                                                             (128, "bf16", 8, 4, 1), (128, "f16", 2, 8, 3), (128, "f16", 6, 12, 1),
                                                             (256, "bf16", 2, 8, 1), (256, "f16", 1, 5, 2)])
@pytest.mark.parametrize("lens", [[1537], [0, 0, 1602, 0], [1] * 40 + [1999], [4000, 3999]])
def test_long_rows_take_shares(gvr, workspace, dim, dtype, kv_heads, group, next_n, lens):  # noqa: F811
    decode_case(gvr, dim + len(lens), dim, dtype, kv_heads, group, 16, next_n, 1, lens, 0, pages=80)
    assert written(workspace)


@pytest.mark.parametrize("requests,shares", [(150, True), (301, True), (1024, True), (1025, False)])
def test_many_rows_take_shares_up_to_a_number(gvr, workspace, requests, shares):  # noqa: F811
    lens = np.random.default_rng(requests).integers(0, 20, requests)
    lens[requests // 3] = 1600
    decode_case(gvr, requests, 64, "bf16", 1, 2, 32, 1, 1, lens, 0, pages=60)
    assert written(workspace) == shares


@pytest.mark.parametrize("lens,k,shares", [([1500], 0, False), ([9500, 700], 2048, False), ([9500, 700], 2049, True),
                                           ([9500, 700, 8200], 9001, True)])
def test_short_rows_and_selections_take_clusters(gvr, workspace, lens, k, shares):  # noqa: F811
    decode_case(gvr, k, 64, "bf16", 2, 3, 16, 1, 1, lens, k)
    assert written(workspace) == shares


def test_a_workspace_without_room_is_not_written(gvr, workspace, monkeypatch):  # noqa: F811
    from sparse_attention_indexer_exact_gb300 import cache as mod
    monkeypatch.setattr(mod, "_WORKSPACE", 1000)
    decode_case(gvr, 3, 128, "bf16", 8, 4, 16, 1, 1, [4000], 0, pages=90)
    assert not written(workspace)
