"""Build libmuonclip.so (in-tree) for sm_103a with nvcc.

Each translation unit is compiled in parallel, then linked against the shared
CUDA runtime.  Beside it the binding's helper module _host.so (host code) is
compiled against torch's headers and linked to the library.  Both are rebuilt
only when a source or header is newer, or torch is another version.  Run as ``python -m muon_qk_clip_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmuonclip.so")
HOST = os.path.join(PKG, "_host.so")
HOST_SRC = os.path.join(CSRC, "host.cxx")
HOST_TORCH = os.path.join(BUILD, "host.torch")         # the torch that _host.so was compiled against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def cuda_lib_dir() -> str:
    base = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    for sub in ("lib64", "lib", "targets/sbsa-linux/lib", "targets/x86_64-linux/lib"):
        d = os.path.join(base, sub)
        if os.path.exists(os.path.join(d, "libcudart.so")):
            return d
    return os.path.join(base, "lib64")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(HOST) or not os.path.exists(HOST_TORCH):
        return True
    with open(HOST_TORCH) as f:
        if f.read() != importlib.metadata.version("torch"):
            return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(HOST))
    deps = sources() + [HOST_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
           "--expt-relaxed-constexpr", "-I", INCLUDE, "-c", src, "-o", obj, *extra]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_host() -> str:
    import torch
    home = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "host.o")
    cmd = [_gxx(), "-O2", "-std=c++17", "-fPIC", "-c", "-I", os.path.join(home, "include"),
           "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(os.path.dirname(cuda_lib_dir()), "include"),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", HOST_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(HOST_SRC)}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_host(obj: str):
    import torch
    home = os.path.dirname(torch.__file__)
    tmp = HOST + ".tmp"
    cmd = [_gxx(), "-shared", "-o", tmp, obj, "-L", PKG, "-l:libmuonclip.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-L", cuda_lib_dir(), f"-Wl,-rpath-link,{cuda_lib_dir()}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _host.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, HOST)
    with open(HOST_TORCH, "w") as f:
        f.write(importlib.metadata.version("torch"))


def _gxx() -> str:
    return shutil.which("g++") or "g++"


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile every source for sm_103a, link libmuonclip.so, and build _host.so;
    returns the library's path."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        host = ex.submit(_compile_host)
        objs = list(ex.map(lambda s: _compile(s, list(extra)), srcs))
        host_obj = host.result()
    libdir = cuda_lib_dir()
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-L", libdir, "-lcudart",
           "-Xlinker", f"-rpath,{libdir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_host(host_obj)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
