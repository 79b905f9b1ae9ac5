"""The cache calls' sources and bindings, on the host: what a GPU test could not show, or could show only by a fault."""
from __future__ import annotations

import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_attention_indexer_exact_gb300")


def code(path):
    """The source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(PKG, "csrc_cache", "*"))), ids=os.path.basename)
def test_nothing_is_read_as_read_only(path):
    """The kernels can be resident while the one before them still writes their inputs, so no load may take the
    read-only path, nor a pointer promise that nothing else writes there."""
    assert not re.findall(r"__ldg\w*|ld\.global\.nc|__restrict__", code(path))


def test_every_kernel_waits_for_the_one_before_it():
    """Each __global__ function has begin() in its body (join_kernel after the lengths, which the kernel before it read)."""
    kernels = 0
    for path in glob.glob(os.path.join(PKG, "csrc_cache", "*.cu*")):
        for body in re.split(r"__global__", code(path))[1:]:
            kernels += 1
            assert re.search(r"\bbegin\(\);", body.split("\n}\n")[0])
    assert kernels == 6


# ------------------------------------------------------------------------------------- arguments
@pytest.fixture(scope="module")
def gvr():
    from sparse_attention_indexer_exact_gb300 import _build
    _build.build_library()
    import sparse_attention_indexer_exact_gb300 as mod
    mod.load_library()
    return mod


@pytest.mark.parametrize("beyond", [2 ** 31, 2 ** 32 + 1, -2 ** 31 - 1, 2 ** 70])
def test_integers_beyond_32_bits_are_refused(gvr, beyond):
    """Cut to 32 bits they would be other numbers: 2^32 + 1 draft rows would read a length for each row where one was
    given for all.  (The host's tensors come to their own refusal only behind this one.)"""
    torch = pytest.importorskip("torch")
    i32 = torch.zeros(3, dtype=torch.int32)
    cache, table, x = torch.zeros(4, 16, 2, 144, dtype=torch.uint8), i32[:, None], torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="head_dim"):
        gvr.cache_row_bytes(beyond)
    with pytest.raises(ValueError, match="page_size"):
        gvr.cache_tables(i32, i32, i32, table, 5, beyond)
    with pytest.raises(ValueError, match="compress_ratio"):
        gvr.cache_tables(i32, i32, i32, table, 5, 16, beyond)
    with pytest.raises(ValueError, match="next_n"):
        gvr.attend_decode(x, cache, table, i32, beyond, 1)
    with pytest.raises(ValueError, match="compress_ratio"):
        gvr.attend_decode(x, cache, table, i32, 1, beyond)


def test_integers_of_other_types_are_taken_and_fractions_refused(gvr):
    np = pytest.importorskip("numpy")
    assert gvr.cache_row_bytes(np.int64(128)) == 144
    with pytest.raises(TypeError):
        gvr.cache_row_bytes(128.0)


def test_tables_of_too_many_elements_are_refused(gvr):
    """8192 requests of 2^18 pages each could take 2^31 new ones, which sums of 32 bits do not tell apart."""
    lib, at, missing, argument = gvr.load_library(), 0x10000, 1, 5  # an aligned address that is never read

    def call(requests, width):  # without counts, so refused in any case, behind the check of the sizes
        return lib.cache_tables(at, at, requests, 1, 1, at, 9, at, width, width, at, 40, None, None)

    for requests, width in ((8192, 2 ** 18), (8191, 2 ** 18 + 65), (2, 2 ** 30), (8192, 2 ** 31 - 1)):
        assert requests * width >= 2 ** 31 and call(requests, width) == argument
    for requests, width in ((8192, 2 ** 18 - 1), (1, 2 ** 31 - 1), (0, 2 ** 31 - 1)):
        assert requests * width < 2 ** 31 and call(requests, width) == missing
