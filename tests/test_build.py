"""build.py on a host where the Python extension cannot be built."""
import ctypes
import os
import subprocess

import pytest

from stage_software_pipelining_gb300 import build as gemm_build


@pytest.fixture
def small_build(tmp_path, monkeypatch):
    """build() with one small C source in place of the kernels, in a directory of its own."""
    src = tmp_path / "answer.c"
    src.write_text("int answer(void) { return 42; }\n")

    def compile_c(path, verbose):
        obj = str(tmp_path / "answer.o")
        subprocess.run(["gcc", "-fPIC", "-c", path, "-o", obj], check=True)
        return obj

    monkeypatch.setattr(gemm_build, "LIB", str(tmp_path / "libgemm.so"))
    monkeypatch.setattr(gemm_build, "BINDING", str(tmp_path / "_quant.so"))
    monkeypatch.setattr(gemm_build, "OUT_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(gemm_build, "sources", lambda: [str(src)])
    monkeypatch.setattr(gemm_build, "_compile", compile_c)
    return tmp_path


def missing():
    raise RuntimeError("no Python.h here")


def test_library_is_linked_without_the_extension(small_build, monkeypatch):
    monkeypatch.setattr(gemm_build, "_compile_binding", missing)
    with pytest.raises(RuntimeError, match="_quant.so.*no Python.h here"):
        gemm_build.build(force=True)
    assert ctypes.CDLL(str(small_build / "libgemm.so")).answer() == 42
    assert not os.path.exists(small_build / "_quant.so")


def test_missing_torch_is_named(small_build, monkeypatch):
    import importlib.util
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    with pytest.raises(RuntimeError, match="torch is not installed"):
        gemm_build.build(force=True)
    assert os.path.exists(small_build / "libgemm.so")
