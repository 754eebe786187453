"""The C library is built and the paged helpers work where the CPython binding cannot be:
without torch or a compiler at build time, or with a binding for another torch."""
import builtins
import os
import shutil
import subprocess
import types
import warnings

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
from exact_attention_blackwell_gb300 import build as fa_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()


def test_it_is_built_and_loaded_here():
    assert os.path.exists(fa_build.build_binding())
    assert fa._paged_binding().__name__ == "_paged_binding" and callable(fa._paged_binding().attention)


def test_each_interpreter_and_torch_has_its_own(monkeypatch):
    names = set()
    for abi in (".cpython-312-x86_64-linux-gnu.so", ".cpython-313-x86_64-linux-gnu.so", ".cpython-312-aarch64-linux-gnu.so"):
        for version in ("2.9.1+cu130", "2.11.0+cu130"):
            monkeypatch.setattr(fa_build.sysconfig, "get_config_var", lambda name: abi)
            path = fa_build.binding_path(types.SimpleNamespace(__version__=version))
            assert path.endswith(abi)
            names.add(path)
    assert len(names) == 6


def without_torch(monkeypatch):
    real = builtins.__import__

    def no_torch(name, *a, **kw):
        if name == "torch" or name.startswith("torch."):
            raise ImportError("no torch here")
        return real(name, *a, **kw)

    monkeypatch.setattr(builtins, "__import__", no_torch)


def test_the_library_needs_no_torch(monkeypatch):
    without_torch(monkeypatch)
    assert fa_build.build_binding() is None and fa_build.build_binding(force=True) is None
    assert fa_build.build() == fa_build.LIB_PATH  # up to date


def test_the_library_is_built_without_torch(monkeypatch, tmp_path):
    """From the start, with the compiler's work left out: what build() asks for and where it puts it."""
    asked = []

    def run(cmd, **kw):
        asked.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    path = str(tmp_path / "lib.so")
    monkeypatch.setattr(fa_build, "LIB_PATH", path)
    monkeypatch.setattr(fa_build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(fa_build.subprocess, "run", run)
    without_torch(monkeypatch)
    assert fa_build.build(lib_path=path) == path and os.path.exists(path)
    assert asked and not any(fa_build.BINDING_SRC in cmd for cmd in asked)


def test_no_compiler_or_headers_no_binding(monkeypatch, tmp_path):
    monkeypatch.setattr(fa_build, "binding_path", lambda t: str(tmp_path / "none.so"))
    with monkeypatch.context() as m:
        m.delenv("CXX", raising=False)
        m.setattr(shutil, "which", lambda name: None)
        m.setattr(fa_build, "nvcc_path", lambda: "/usr/local/cuda/bin/nvcc")
        assert fa_build.build_binding() is None
    with monkeypatch.context() as m:
        m.setattr(fa_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
        assert fa_build.build_binding() is None


def test_a_binding_that_does_not_compile_leaves_the_library(monkeypatch, tmp_path):
    def run(cmd, **kw):
        if fa_build.BINDING_SRC in cmd:
            return subprocess.CompletedProcess(cmd, 1, "", "no such member")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    path = str(tmp_path / "lib.so")
    monkeypatch.setattr(fa_build, "LIB_PATH", path)
    monkeypatch.setattr(fa_build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(fa_build, "binding_path", lambda t: str(tmp_path / "none.so"))
    monkeypatch.setattr(fa_build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="no such member"):
        fa_build.build(lib_path=path)
    assert os.path.exists(path)


@pytest.fixture(params=["missing", "broken"])
def no_binding(request, monkeypatch, tmp_path):
    path = tmp_path / "binding.so"
    if request.param == "broken":
        path.write_bytes(b"not a library")
    monkeypatch.setattr(fa, "_fast", None)
    monkeypatch.setattr(fa_build, "binding_path", lambda t: str(path))


def test_without_a_binding_the_helpers_still_check(no_binding):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="ctypes"), pytest.raises(ValueError, match="CUDA"):
        fa.cache_fork(i32(9), i32(3, 4), i32(3), i32(3), 16)
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # it is said once
        with pytest.raises(ValueError, match="CUDA"):
            fa.cache_fork(i32(9), i32(3, 4), i32(3), i32(3), 16)


@pytest.mark.gpu
def test_without_a_binding_the_calls_are_made(no_binding):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    refs, table = i32([1, 1, 1, 0]), i32([[0, 1], [2, -1]])
    with pytest.warns(RuntimeWarning, match="ctypes"):
        lens = fa.cache_fork(refs, table, i32([20, 3]), i32([0, 0]), 16)
    assert lens.tolist() == [20, 20] and table.tolist() == [[0, 1], [0, 1]] and refs.tolist() == [2, 2, 0, 0]
    k = torch.randn((4, 16, 2, 64), device="cuda").to(torch.bfloat16)
    lens, status = fa.cache_resize(refs, k, k.clone(), table, lens, i32([21, 20]))
    assert lens.tolist() == [21, 20] and status.tolist() == [0, 0] and table.tolist() == [[0, 2], [0, 1]]
