"""The build: the C library does not need its Python binding, nor torch.

Each test builds a little source tree of its own, in a process of its own.
"""
import ctypes
import importlib.util
import os
import subprocess
import sys

import pytest

from paged_kv_cache_172_gb300 import build_lib

PRELUDE = """
import importlib.util, os, sys
at = sys.argv[1]
{before}
spec = importlib.util.spec_from_file_location("build_lib", {path!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.PKG = at
b.CSRC = os.path.join(at, "csrc")
b.OBJ_DIR = os.path.join(at, "_build")
b.LIB = os.path.join(at, "libpagedkv.so")
b.BINDING = os.path.join(at, "_grouped.so")
b.build()
"""


def run(at, before=""):
    code = PRELUDE.format(before=before, path=build_lib.__file__)
    return subprocess.run([sys.executable, "-c", code, str(at)], capture_output=True, text=True)


@pytest.fixture
def tree(tmp_path):
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").write_text('extern "C" int answer() { return 42; }\n')
    (tmp_path / "csrc" / "py_grouped.cpp").write_text("int nothing;\n")
    return tmp_path


def check_library(tree):
    assert ctypes.CDLL(str(tree / "libpagedkv.so")).answer() == 42


def test_library_is_built_without_torch(tree):
    r = run(tree, before="sys.modules['torch'] = None  # not to be imported")
    assert r.returncode == 0, r.stderr
    check_library(tree)
    assert not (tree / "_grouped.so").exists()
    assert "torch" in r.stderr and "binding" in r.stderr  # it says what is missing


def test_library_is_linked_where_the_binding_does_not_compile(tree):
    (tree / "_grouped.so").write_bytes(b"an older one")
    (tree / "csrc" / "py_grouped.cpp").write_text("#error broken on purpose\n")
    r = run(tree)
    assert r.returncode != 0
    assert "g++" in r.stderr and "broken on purpose" in r.stderr and "nvcc failed" not in r.stderr
    check_library(tree)
    assert not (tree / "_grouped.so").exists()  # a binding of other sources does not stay


def test_binding_follows_torch(tree):
    # the same place, another version: what was compiled against the older one is not kept
    real = os.path.dirname(importlib.util.find_spec("torch").origin)
    fake = tree / "site" / "torch"
    (fake / "include").mkdir(parents=True)
    (fake / "lib").symlink_to(os.path.join(real, "lib"))
    (fake / "__init__.py").write_text("")
    obj = tree / "_build" / "py_grouped.o"
    before = "sys.path.insert(0, os.path.join(at, 'site'))"
    times = []
    for version in ("2.9.1", "2.9.1", "2.11.0"):
        (fake / "version.py").write_text(f"__version__ = {version!r}\n")
        r = run(tree, before=before)
        assert r.returncode == 0, r.stderr
        times.append((obj.stat().st_mtime_ns, (tree / "_grouped.so").stat().st_mtime_ns))
    assert times[0] == times[1]
    assert times[2][0] > times[1][0] and times[2][1] > times[1][1]
    check_library(tree)
