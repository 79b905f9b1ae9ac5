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
