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
