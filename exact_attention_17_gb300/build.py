"""Compile libfa2.so (sm_103a) in-tree with nvcc, and the torch binding with g++.

The kernel families live in separate translation units that compile in
parallel; the host side links the CUDA runtime statically and finds the
driver entry points it needs (tensor-map encoding, address ranges) at run
time, so the library has no link-time dependency on libcuda.  The binding
(_binding.so) is a Python extension module against torch's headers and is
handed the library's functions when it is loaded.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libfa2.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["fa2_api.cu", "fa2_tc_d64_bf16.cu", "fa2_tc_d128_bf16.cu", "fa2_tc_d256_bf16.cu",
           "fa2_tc_d64_f16.cu", "fa2_tc_d128_f16.cu", "fa2_tc_d256_f16.cu", "fa2_simt.cu",
           "fa2_combine.cu", "fa2_bwd.cu", "fa2_tc_pair_d128.cu", "fa2_bwd2.cu",
           "fa2_paged_api.cu", "fa2_paged_bf16.cu", "fa2_paged_f16.cu", "fa2_rope.cu", "fa2_pages.cu"]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    files += glob.glob(os.path.join(INCLUDE, "*.h"))
    return files


def _newer(path, files):
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in files)


def up_to_date() -> bool:
    return os.path.exists(LIB_PATH) and _newer(LIB_PATH, _inputs())


def _replace(path, make):
    """Has make(temporary path) write a file next to `path`, then puts it in its place."""
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=PKG)
    os.close(fd)
    try:
        r = subprocess.run(make(tmp), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"building {os.path.basename(path)} failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, path)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)


def build_binding(force: bool = False) -> str | None:
    """Build _binding.so unless it is newer than its sources and the torch it is built against.

    Returns its path, or None where something that it alone needs is not there:
    torch with its headers and CUDA libraries, Python's headers, g++.  The
    library works without it (paged.py then goes through ctypes).
    """
    spec = importlib.util.find_spec("torch")   # found, not imported
    torch_dir = os.path.dirname(spec.origin) if spec is not None and spec.origin else None
    sources = [BINDING_SOURCE, os.path.join(INCLUDE, "fa2.h")]
    python_include = sysconfig.get_paths()["include"]
    needed = [os.path.join(python_include, "Python.h")]
    if torch_dir is not None:
        libs = os.path.join(torch_dir, "lib")
        needed += [os.path.join(libs, "libtorch_python.so"), os.path.join(libs, "libc10_cuda.so"),
                   os.path.join(torch_dir, "include", "ATen", "core", "Tensor.h")]
    there = os.path.exists(BINDING_PATH)
    if torch_dir is None or shutil.which("g++") is None or not all(os.path.exists(f) for f in needed):
        if there and not _newer(BINDING_PATH, sources):
            os.remove(BINDING_PATH)            # made for another interface of the library
        return None
    if not force and there and _newer(BINDING_PATH, sources + [os.path.join(torch_dir, "version.py")]):
        return BINDING_PATH
    includes = [INCLUDE, os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                python_include, os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    _replace(BINDING_PATH, lambda tmp: ["g++", "-O2", "-std=c++17", "-fPIC", "-shared"] + ["-I" + i for i in includes]
             + [BINDING_SOURCE, "-o", tmp, "-L" + libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                "-Wl,-rpath," + libs])
    return BINDING_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libfa2.so and, where torch is there, the binding next to this file unless they are newer than their
    sources."""
    if not force and up_to_date():
        build_binding()
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I" + INCLUDE, "-I" + CSRC]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc()] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding, force)
        results = list(ex.map(compile_one, SOURCES))
        binding.result()
    if verbose:
        for _, log in results:
            print(log)
    _replace(LIB_PATH, lambda tmp: [nvcc()] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results])
    return LIB_PATH


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
