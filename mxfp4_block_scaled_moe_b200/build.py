"""Build libmxfp4moe.so (the CUDA library behind include/mxfp4_moe.h) for sm_100a.

Every .cu file under csrc/ is compiled by nvcc with
``-gencode arch=compute_100a,code=sm_100a -O3 -lineinfo`` (no fast-math: IEEE division
and square roots, no flush-to-zero) and linked into one shared library with the CUDA
runtime linked statically. The library lands next to this file, inside the package.

csrc/host_ops.cpp, the operators' native host side, becomes the Python extension
_host_ops.so beside it (compiled by g++ against the installed torch). The library does not
need it: without torch it is left out, and where it cannot be compiled the library is
linked before that is raised. It carries the torch and Python it was compiled for and is
compiled anew for others.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "mxfp4moe")
LIB = os.path.join(HERE, "libmxfp4moe.so")
HOST_OPS = os.path.join(HERE, "_host_ops.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xptxas", "-warn-spills", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(lib, deps):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps)


def host_ops_abi() -> str:
    """What host_ops.cpp is compiled for; the extension holds it as `built_for`."""
    import torch
    return f"torch {torch.__version__}, python {sys.version_info.major}.{sys.version_info.minor}"


def _built_for(path, abi):
    with open(path, "rb") as f:
        return b"built for: " + abi.encode() + b"\0" in f.read()


def build_host_ops(force: bool = False) -> str:
    src = os.path.join(CSRC, "host_ops.cpp")
    abi = host_ops_abi()
    if not force and not _stale(HOST_OPS, [src, os.path.join(INCLUDE, "mxfp4_moe.h"), __file__]) \
            and _built_for(HOST_OPS, abi):
        return HOST_OPS
    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = cpp_extension.include_paths() + [os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = f"{HOST_OPS}.{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DMXMOE_BUILT_FOR="{abi}"',
           *[a for i in inc for a in ("-isystem", i)],
           src, "-o", tmp, "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, HOST_OPS)
    return HOST_OPS


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    srcs = sources()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "mxfp4_moe.h"))
    host_ops = importlib.util.find_spec("torch") is not None
    if not force and not _stale(LIB, srcs + headers + [__file__]):
        if host_ops:
            build_host_ops()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        host = ex.submit(build_host_ops, force) if host_ops else None
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if host is not None:
        host.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
