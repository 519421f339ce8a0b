"""The CUDA library builds by itself: without torch, and whatever becomes of the Python binding."""
import os
import subprocess
import sys

import pytest

from dense_tensor_core_gb300 import build as b


@pytest.fixture
def small(tmp_path, monkeypatch):
    """build() with a library of one small source, into a folder of its own."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(b, "sources", lambda: [str(src)])
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libdtc_gemm.so"))
    monkeypatch.setattr(b, "NATIVE", str(tmp_path / "_ffn_native.so"))
    monkeypatch.setattr(b, "OBJ_DIR", str(tmp_path / "obj"))
    return src


def test_without_torch(small, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # an import of torch fails
    assert b.build() == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.NATIVE)
    before = os.stat(b.LIB).st_mtime_ns
    assert b.build() == b.LIB and os.stat(b.LIB).st_mtime_ns == before  # nothing is left to do


def test_binding_that_does_not_compile_leaves_the_library(small, monkeypatch):
    def broken(obj_dir):
        raise subprocess.CalledProcessError(1, "g++")

    monkeypatch.setattr(b, "_compile_native", broken)
    with pytest.raises(subprocess.CalledProcessError):  # (reported)
        b.build()
    assert os.path.exists(b.LIB)
    before = os.stat(b.LIB).st_mtime_ns
    with pytest.raises(subprocess.CalledProcessError):
        b.build()
    assert os.stat(b.LIB).st_mtime_ns == before


def test_each_is_made_again_for_its_own_sources(small, monkeypatch):
    made = []
    monkeypatch.setattr(b, "_compile_native", lambda d: made.append("object"))
    monkeypatch.setattr(b, "_link_native", lambda obj, tmp: (made.append("module"), open(tmp, "w").close()))
    b.build()
    assert made == ["object", "module"]
    os.utime(small, ns=(os.stat(b.LIB).st_mtime_ns + 10 ** 9,) * 2)  # the kernels are newer
    lib = os.stat(b.LIB).st_ino
    b.build()
    assert made == ["object", "module"] and os.stat(b.LIB).st_ino != lib
