"""Build the CUDA library in-tree: ``paged_kv_cache_151_gb300/_build/libpa.so``.

Every translation unit under ``csrc/`` is compiled in parallel -- the CUDA
units (``.cu``) for sm_103a only (``-gencode arch=compute_103a,code=sm_103a``),
the host-only units (``.cpp``: the block manager) by nvcc's host compiler --
then linked into one shared library exporting the C ABI of ``include/*.h``.  Beside it the
Python binding's checks of tensors, ``_build/_tensors.so``, are compiled against the headers
of the torch that is installed.  A unit is rebuilt when it, a header it may include, or the
flags changed.

    python -m paged_kv_cache_151_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import hashlib
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB_NAME = "libpa.so"
LIB_PATH = os.path.join(BUILD, LIB_NAME)

TENSORS_SRC = os.path.join(HERE, "binding", "tensors.cpp")
TENSORS_PATH = os.path.join(BUILD, "_tensors.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-O2", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return sorted(hs)


def _digest(src: str, flags) -> str:
    h = hashlib.sha256()
    for path in [src] + _headers():
        with open(path, "rb") as f:
            h.update(f.read())
    h.update(" ".join(flags).encode())
    return h.hexdigest()


def _compile(src_name: str, force: bool, verbose: bool, extra, out_dir: str) -> str:
    src = os.path.join(CSRC, src_name)
    obj = os.path.join(out_dir, os.path.splitext(src_name)[0] + ".o")
    flags = ARCH + NVCC_FLAGS + list(extra)
    stamp = obj + ".sha"
    dig = _digest(src, flags)
    if not force and os.path.exists(obj) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == dig:
                return obj
    cmd = [nvcc()] + flags + ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src_name}:\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr, flush=True)
    with open(stamp, "w") as f:
        f.write(dig)
    return obj


def build_tensors(force: bool = False) -> str:
    """Compile the binding's checks of tensors; returns the extension's path."""
    import sysconfig

    import torch
    os.makedirs(BUILD, exist_ok=True)
    base = os.path.join(os.path.dirname(torch.__file__))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], TENSORS_SRC,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    with open(TENSORS_SRC, "rb") as f:
        dig = hashlib.sha256(f.read() + " ".join(cmd + [torch.__version__, sys.version]).encode())
    stamp = TENSORS_PATH + ".sha"
    if not force and os.path.exists(TENSORS_PATH) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == dig.hexdigest():
                return TENSORS_PATH
    tmp = TENSORS_PATH + f".tmp{os.getpid()}"
    res = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on tensors.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, TENSORS_PATH)
    with open(stamp, "w") as f:
        f.write(dig.hexdigest())
    return TENSORS_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=(), out_dir: str = None) -> str:
    """Compile and link the library; returns its path.  ``out_dir`` builds a
    separate copy (for example with extra -D flags) instead of the default."""
    out_dir = BUILD if out_dir is None else out_dir
    lib_path = os.path.join(out_dir, LIB_NAME)
    os.makedirs(out_dir, exist_ok=True)
    srcs = _sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        tensors = ex.submit(build_tensors, force)
        objs = list(ex.map(lambda s: _compile(s, force, verbose, extra_flags, out_dir), srcs))
        tensors.result()
    newest = max(os.path.getmtime(o) for o in objs)
    if force or not os.path.exists(lib_path) or os.path.getmtime(lib_path) < newest:
        tmp = lib_path + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, lib_path)
    return lib_path


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true",
                    help="print registers / spills per kernel (-Xptxas -v)")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    path = build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info,
                 extra_flags=extra)
    print(path)


if __name__ == "__main__":
    sys.exit(main())
