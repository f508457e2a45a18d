"""The in-tree build where a compiler fails (no GPU): the C library does not depend on the Python
extension, and an error names the compiler that it comes from."""
import os
import warnings

import pytest

import block_quantized_decode_quantize_gb300 as mem
from block_quantized_decode_quantize_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmemra.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_memra_binding.so"))
    return tmp_path


def compiler(path, status):
    path.write_text("#!/bin/sh\necho no such header\nexit %d\n" % status)
    path.chmod(0o755)
    return str(path)


def test_the_library_is_there_without_the_extension(tree, monkeypatch):
    monkeypatch.setenv("CXX", compiler(tree / "cxx", 1))
    with pytest.warns(RuntimeWarning, match="no such header") as said:
        assert build.build() == build.LIB
    assert "nvcc" not in str(said[0].message) and build.os.environ["CXX"] in str(said[0].message)
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    made = os.path.getmtime(build.LIB)
    with pytest.warns(RuntimeWarning):
        build.build()                                    # tries the extension again, leaves the library
    assert os.path.getmtime(build.LIB) == made


def test_a_compiler_that_is_not_there(tree, monkeypatch):
    monkeypatch.setenv("CXX", str(tree / "none"))
    with pytest.warns(RuntimeWarning, match="none"):
        build.build()
    assert os.path.exists(build.LIB)


def test_a_kernel_that_does_not_compile(tree, monkeypatch):
    monkeypatch.setenv("CXX", compiler(tree / "cxx", 1))
    (tree / "one.cu").write_text("not C++\n")
    with warnings.catch_warnings(), pytest.raises(RuntimeError, match="nvcc failed"):
        warnings.simplefilter("error")
        build.build()
    assert not os.path.exists(build.LIB)


def test_calls_without_the_extension_take_the_long_way(tmp_path, monkeypatch):
    monkeypatch.setattr(mem, "_fast", None)
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "none.so"))
    if not os.path.exists(build.LIB):
        build.build()
    with pytest.warns(RuntimeWarning, match="none.so"):
        quick = mem._binding()
    assert all(getattr(quick, name)(1, 2, 3) is None for name in ("plan", "append", "read", "attention", "route"))
    with warnings.catch_warnings():
        warnings.simplefilter("error")                   # said once
        with pytest.raises(ValueError, match="ctx_lens"):
            mem.memra_kv_plan(1, 2, 16, 3, 4, 5)
