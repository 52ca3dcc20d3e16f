"""Builds libkvq.so in-tree with nvcc for sm_103a (GB300), and kvq_native.so, the torch binding of its serving-step calls.

Each translation unit of csrc/ is compiled by its own nvcc process (in parallel), then linked
into quantized_paged_kv_int4_gb300/libkvq.so against the shared CUDA runtime (the one torch
loads). Objects go to quantized_paged_kv_int4_gb300/_build/. A build is skipped when the
library is newer than every source and header. kvq_native.so (native/binding.cpp, host C++) is linked
against the installed torch and libkvq.so, and built again for another torch or Python.
"""

import importlib.metadata
import importlib.util

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkvq.so")
NATIVE_SRC = os.path.join(PKG, "native", "binding.cpp")
NATIVE = os.path.join(PKG, "kvq_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkvq")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "kvq.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _native_versions():
    return "torch %s python %s" % (importlib.metadata.version("torch"), sys.version)


def native_up_to_date():
    stamp = os.path.join(OBJ, "kvq_native.versions")
    if not os.path.exists(NATIVE) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        if f.read() != _native_versions():
            return False
    t = os.path.getmtime(NATIVE)
    return all(os.path.getmtime(f) <= t for f in (NATIVE_SRC, os.path.join(ROOT, "include", "kvq.h"), os.path.abspath(__file__)))


def _compile_native():
    """native/binding.cpp -> _build/kvq_native.o"""
    torch_dir = list(importlib.util.find_spec("torch").submodule_search_locations)[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj = os.path.join(OBJ, "kvq_native.o")
    os.makedirs(OBJ, exist_ok=True)
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", NATIVE_SRC, "-o", obj,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"),
           "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (NATIVE_SRC, r.stdout, r.stderr))
    return obj


def build_native(force=False, obj=None):
    """Link kvq_native.so (libkvq.so has to be there); returns its path."""
    if not force and native_up_to_date():
        return NATIVE
    obj = obj or _compile_native()
    torch_lib = os.path.join(list(importlib.util.find_spec("torch").submodule_search_locations)[0], "lib")
    tmp = NATIVE + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", LIB, "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of kvq_native.so failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, NATIVE)
    with open(os.path.join(OBJ, "kvq_native.versions"), "w") as f:
        f.write(_native_versions())
    return NATIVE


def build(force=False, verbose=False, ptxas_info=False):
    """Compile csrc/*.cu and link libkvq.so and kvq_native.so; returns libkvq's path."""
    if not force and up_to_date():
        build_native()
        return LIB
    nvcc = _nvcc()
    os.makedirs(OBJ, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        native = None if native_up_to_date() and not force else ex.submit(_compile_native)
        results = list(ex.map(compile_one, sources()))
    if verbose or ptxas_info:
        for obj, log in results:
            if log.strip():
                sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-soname=libkvq.so", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    build_native(force=native is not None, obj=native.result() if native is not None else None)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
