"""In-tree build of libqsa.so for sm_103a (nvcc only; no cmake, no torch extension) and of qsa_torch.so.

Each .cu file under csrc/ compiles to an object in parallel, then nvcc links the
shared library next to this file. Objects go to <repo>/_build (git-ignored). csrc/torch_binding.cpp
(the Python marshalling of the calls that run once per layer) compiles beside them with the host
compiler against the headers of the installed torch, and links to libqsa.so.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(HERE, "libqsa.so")
TORCH_SRC = os.path.join(CSRC, "torch_binding.cpp")
TORCH_PATH = os.path.join(HERE, "qsa_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                 "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA 13 on PATH)")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [TORCH_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _compile(src: str, verbose: bool, ptxas_v: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [nvcc()] + CFLAGS + (["-Xptxas", "-v"] if ptxas_v else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or ptxas_v or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
    return obj


def _compile_torch(verbose: bool) -> str:
    """torch_binding.cpp -> an object (torch's headers are found, nothing of torch is run)."""
    import importlib.util
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    obj = os.path.join(BUILD_DIR, "torch_binding.cpp.o")
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"]
    cmd += [a for i in includes for a in ("-isystem" if "torch" in i else "-I", i)] + ["-c", TORCH_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("the host compiler failed on torch_binding.cpp")
    return obj


def _link_torch(obj: str, verbose: bool) -> None:
    import importlib.util
    lib_dir = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
    tmp = TORCH_PATH + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", HERE, "-l:libqsa.so", "-L", lib_dir,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,--allow-shlib-undefined"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("the link of qsa_torch.so failed")
    os.replace(tmp, TORCH_PATH)


def build(verbose: bool = False, force: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every CUDA source and link libqsa.so; returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    newest = max(os.path.getmtime(p) for p in _deps())
    if not force and not ptxas_verbose and all(os.path.exists(p) and os.path.getmtime(p) >= newest
                                               for p in (LIB_PATH, TORCH_PATH)):
        return LIB_PATH
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        torch_obj = ex.submit(_compile_torch, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose, ptxas_verbose), srcs))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("nvcc link of libqsa.so failed")
    os.replace(tmp, LIB_PATH)
    _link_torch(torch_obj.result(), verbose)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, force=True, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB_PATH)
