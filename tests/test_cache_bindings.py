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


# ------------------------------------------------------------------- the library without its tensor binding
@pytest.fixture
def commands(monkeypatch):
    """The commands that a build runs, which are not run."""
    from sparse_attention_indexer_exact_gb300 import _build
    ran = []
    monkeypatch.setattr(_build, "_run", lambda cmd: ran.append(cmd) or "")
    return ran


def lacking(monkeypatch, what):
    from sparse_attention_indexer_exact_gb300 import _build
    if what == "torch":
        find = _build.importlib.util.find_spec
        monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    elif what == "Python's headers":
        monkeypatch.setattr(_build.sysconfig, "get_paths", lambda *a: {"include": os.path.join(ROOT, "none")})
    else:
        monkeypatch.setattr(_build.shutil, "which", lambda name: None)


@pytest.mark.parametrize("what", ["torch", "Python's headers", "g++"])
def test_the_library_is_built_where_its_binding_cannot_be(commands, monkeypatch, what):
    from sparse_attention_indexer_exact_gb300 import _build
    lacking(monkeypatch, what)
    with pytest.warns(RuntimeWarning, match="_native.so is not built"):
        assert _build.build_library(force=True) == _build.LIB_PATH
    assert len(commands) == len(_build.units()) + 1 and _build.LIB_PATH in commands[-1]
    assert not any(_build.NATIVE_SOURCE in c or _build.NATIVE_PATH in c for c in commands)


def test_a_binding_that_does_not_compile_leaves_the_library(monkeypatch):
    from sparse_attention_indexer_exact_gb300 import _build
    ran = []

    def run(cmd):
        if _build.NATIVE_SOURCE in cmd:
            raise RuntimeError("no")
        ran.append(cmd)
        return ""

    monkeypatch.setattr(_build, "_run", run)
    with pytest.raises(RuntimeError):
        _build.build_library(force=True)
    assert _build.LIB_PATH in ran[-1] and len(ran) == len(_build.units()) + 1


def test_cache_calls_without_the_binding_go_step_by_step(gvr, monkeypatch):
    """As far as the host goes: each call comes to the checks that name what is wrong."""
    import sys
    torch = pytest.importorskip("torch")
    from sparse_attention_indexer_exact_gb300 import cache
    monkeypatch.setattr(cache, "_native", None)
    monkeypatch.delattr(gvr, "_native", raising=False)
    monkeypatch.setitem(sys.modules, gvr.__name__ + "._native", None)  # as if the file were not there
    i32, c, x = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 16, 2, 144, dtype=torch.uint8), torch.zeros(3, 2, 128).half()
    with pytest.warns(RuntimeWarning, match="_native.so is missing"):
        with pytest.raises(TypeError, match="CUDA"):
            gvr.cache_append(x, x, c, i32)
    import warnings
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # said once
        for call in (lambda: gvr.cache_tables(i32, i32, i32, i32[:, None], 5, 16), lambda: gvr.cache_read(c, i32, 128),
                     lambda: gvr.attend_decode(x, c, i32[:, None], i32, 1, 1),
                     lambda: gvr.attend_prefill(x, c, i32[:, None], i32, i32, i32, i32[:, None])):
            with pytest.raises(TypeError, match="CUDA"):
                call()


# ----------------------------------------------------------------------- the binding under another torch
def test_the_binding_is_rebuilt_for_another_torch(gvr, commands, monkeypatch, tmp_path):
    from sparse_attention_indexer_exact_gb300 import _build
    _build.build_library()
    assert not commands  # all there
    stamp = tmp_path / "stamp"
    monkeypatch.setattr(_build, "NATIVE_STAMP", str(stamp), raising=False)
    for before in (None, "torch 2.8.0, cpython-312-x86_64-linux-gnu"):
        if before:
            stamp.write_text(before)
        commands.clear()
        _build.build_library()
        assert [_build.NATIVE_SOURCE in c for c in commands] == [True, False]  # compiled and linked, and nothing else
        assert stamp.read_text() == _build.native_target()
    commands.clear()
    _build.build_library()
    assert not commands


def test_the_binding_knows_what_it_was_built_for(gvr):
    torch = pytest.importorskip("torch")
    from sparse_attention_indexer_exact_gb300 import _build, _native
    assert _native.BUILT_FOR == _build.native_target() and f"torch {torch.__version__}," in _native.BUILT_FOR


def test_a_binding_for_another_torch_is_not_used(gvr, monkeypatch):
    """Its file may load, but reads tensors by another layout: the call goes step by step."""
    import sys
    from types import SimpleNamespace
    torch = pytest.importorskip("torch")
    from sparse_attention_indexer_exact_gb300 import cache

    def never(*args):
        raise AssertionError("used")

    other = SimpleNamespace(BUILT_FOR="torch 2.8.0, cpython-312-x86_64-linux-gnu", cache_append=never)
    monkeypatch.setattr(cache, "_native", None)
    monkeypatch.setattr(gvr, "_native", other, raising=False)
    monkeypatch.setitem(sys.modules, gvr.__name__ + "._native", other)
    i32, c, x = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 16, 2, 144, dtype=torch.uint8), torch.zeros(3, 2, 128).half()
    with pytest.warns(RuntimeWarning, match="built for torch 2.8.0"):
        with pytest.raises(TypeError, match="CUDA"):
            gvr.cache_append(x, x, c, i32)


def test_a_binding_that_does_not_say_what_it_was_built_for_is_not_used(gvr, monkeypatch):
    import sys
    from types import SimpleNamespace
    from sparse_attention_indexer_exact_gb300 import cache
    pytest.importorskip("torch")
    monkeypatch.setattr(cache, "_native", None)
    monkeypatch.setattr(gvr, "_native", SimpleNamespace(), raising=False)
    monkeypatch.setitem(sys.modules, gvr.__name__ + "._native", gvr._native)
    with pytest.warns(RuntimeWarning, match="built for an unknown torch"):
        assert cache._short().cache_append() is None


def test_limits_of_attention_stand_in_its_header(gvr):
    """At the header's limits a call comes to the pointer it lacks; beyond them it is refused for its arguments."""
    import ctypes
    from sparse_attention_indexer_exact_gb300.cache import _Cache
    header = open(os.path.join(ROOT, "include", "gvr_cache.h")).read()
    assert "GVR_ATTEND_MAX_NEXT_N 4096\n" in header and "GVR_ATTEND_MAX_HEADS (1 << 20)\n" in header and "1 to 65535 */" in header
    lib, at, missing, argument = gvr.load_library(), 0x10000, 1, 5  # an aligned address that is never read

    def call(next_n=1, heads=4, kv_heads=2):  # without lengths, so refused in any case
        cache = _Cache(at, 10, 16 * kv_heads * 144, 16, kv_heads, 128, 0, 1.0, 1.0)
        return lib.attend_decode(ctypes.byref(cache), at, 512, 128, 0, 4, heads, at, 8, 8, None, next_n, 4, at, 32, 0.1, at, None,
                                 None, 0, None)

    for kw in (dict(next_n=4096), dict(heads=1 << 20), dict(heads=65535, kv_heads=65535)):
        assert call(**kw) == missing, kw
    for kw in (dict(next_n=0), dict(next_n=4097), dict(heads=(1 << 20) + 2), dict(heads=65536, kv_heads=65536)):
        assert call(**kw) == argument, kw
