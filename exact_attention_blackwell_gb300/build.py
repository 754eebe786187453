"""Builds the CUDA library ``libfa_gb300.so`` (in-tree, beside this file).

Every ``csrc/*.cu`` translation unit is compiled for sm_103a only, in parallel,
then linked into one shared library with the CUDA runtime linked statically,
so the C ABI of ``include/fa.h`` is the only interface.  The torch helpers of the
paged cache have their ordinary call in a small CPython module beside it
(``csrc/paged_binding.cpp``), compiled with the host compiler against the
installed torch, where there is one, and named after its version and Python's ABI.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import re
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libfa_gb300.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
                   f"-I{CSRC}", f"-I{os.path.join(os.path.dirname(HERE), 'include')}"] + list(extra)


BINDING_SRC = os.path.join(CSRC, "paged_binding.cpp")


def binding_path(torch) -> str:
    """Named after torch's version and the interpreter's ABI: it is compiled against both."""
    abi = sysconfig.get_config_var("EXT_SUFFIX") or ".so"
    return os.path.join(HERE, "_paged_binding_" + re.sub(r"[^0-9A-Za-z]", "_", torch.__version__) + abi)


def build_binding(force: bool = False) -> str | None:
    """Path of the binding, or None where it cannot be built: no torch with CUDA, its headers, Python's, or a host
    compiler.  The C library needs none of them, and without the binding the helpers call it through ctypes."""
    try:
        import torch
    except ImportError:
        return None
    path = binding_path(torch)
    header = os.path.join(os.path.dirname(HERE), "include", "fa.h")
    if not force and os.path.exists(path) and os.path.getmtime(path) >= max(map(os.path.getmtime, (BINDING_SRC, header))):
        return path
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")
    libs, include, python = os.path.join(root, "lib"), os.path.join(root, "include"), sysconfig.get_paths()["include"]
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    needs = (os.path.join(include, "torch", "csrc", "autograd", "python_variable.h"), os.path.join(python, "Python.h"),
             os.path.join(libs, "libc10_cuda.so"))
    if not cxx or not all(map(os.path.exists, needs)):
        return None
    tmp = path + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{include}",
           f"-I{os.path.join(include, 'torch', 'csrc', 'api', 'include')}", f"-I{python}",
           f"-I{cuda}", BINDING_SRC, "-o", tmp, f"-L{libs}", f"-Wl,-rpath,{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, extra_flags=(), lib_path: str = LIB_PATH) -> str:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [
        os.path.join(os.path.dirname(HERE), "include", "fa.h")]
    newest = max(os.path.getmtime(p) for p in deps)
    if not force and not extra_flags and os.path.exists(lib_path) and os.path.getmtime(lib_path) >= newest:
        build_binding()
        return lib_path
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = nvcc_path()
    tag = "x".join(f for f in extra_flags).replace("-", "").replace("=", "") or "default"
    if len(tag) > 64:  # keep object names within the file system's limit
        tag = "v" + hashlib.sha256(tag.encode()).hexdigest()[:16]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + f".{tag}.o")
        cmd = [nvcc] + _flags(extra_flags) + ["-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(build_binding, force) if lib_path == LIB_PATH else None
        objs = list(ex.map(compile_one, srcs))
    tmp = lib_path + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs,
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    if binding is not None:
        binding.result()  # raises where it was compiled and failed; the library is there in any case
    return lib_path


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose="-v" in sys.argv))
