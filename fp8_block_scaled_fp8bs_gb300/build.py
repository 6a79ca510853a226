"""Build libfp8bs.so and _host.so in place: each csrc/*.cu is compiled by nvcc for sm_103a in parallel and
linked into one shared library with the CUDA runtime linked statically (the library depends on
no CUDA shared object at load time; it reaches the driver through the runtime). It needs nvcc and nothing else.
_host.so (csrc/host.cpp) is a CPython module over PyTorch's headers, the host side of the calls that take microseconds:
a step of its own, for the installed PyTorch, and again for another one.

    python -m fp8_block_scaled_fp8bs_gb300.build [--verbose-ptxas] [--library-only]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfp8bs.so")
HOST = os.path.join(PKG, "_host.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              f"-I{os.path.join(ROOT, 'include')}"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the FP8 library needs the CUDA 13 toolkit to build")
    return path


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newest(files):
    return max(os.path.getmtime(f) for f in (*files, os.path.join(ROOT, "include", "fp8bs.h"), os.path.abspath(__file__)))


def up_to_date() -> bool:
    """Of the library alone."""
    sources_ = (os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp"))
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest(sources_)


def _torch_tag() -> str:
    """What _host.so is bound to: PyTorch's C++ interface and the interpreter's."""
    import torch
    return f"torch {torch.__version__} {sys.implementation.cache_tag}\n"


def host_fits() -> bool:
    """Whether there is a _host.so, made for the PyTorch and Python at hand."""
    try:
        with open(HOST + ".txt") as f:
            return os.path.exists(HOST) and f.read() == _torch_tag()
    except OSError:
        return False


def host_up_to_date() -> bool:
    return host_fits() and os.path.getmtime(HOST) >= _newest([os.path.join(CSRC, "host.cpp")])


def build_host() -> str:
    """csrc/host.cpp -> _host.so, with the C++ compiler and the headers and libraries of the installed PyTorch."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler found")
    tmp = HOST + f".tmp{os.getpid()}"
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(f"-I{p}" for p in include_paths()), f"-I{os.path.join(cuda, 'include')}",
           f"-I{sysconfig.get_paths()['include']}", os.path.join(CSRC, "host.cpp"), "-o", tmp,
           *(f"-L{p}" for p in library_paths()), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda",
           "-lc10", "-ldl"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"C++ compiler failed on host.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, HOST)
    with open(tmp, "w") as f:
        f.write(_torch_tag())
    os.replace(tmp, HOST + ".txt")
    return HOST


def _compile(src: str, ptxas_verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if ptxas_verbose:
        sys.stderr.write(res.stderr)
    return obj


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """The library."""
    if not force and not ptxas_verbose and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(lambda s: _compile(s, ptxas_verbose), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs,
           "-Xlinker", "--no-undefined", "-ldl", "-lpthread", "-lrt"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build_all(force: bool = False, ptxas_verbose: bool = False) -> str:
    """The library and, beside it, the host module; the library is there even if the host module fails."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        host = ex.submit(lambda: build_host() if force or not host_up_to_date() else HOST)
        lib = build(force, ptxas_verbose)
        host.result()
    return lib


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--library-only", action="store_true", help="libfp8bs.so alone: needs no PyTorch")
    a = ap.parse_args()
    print((build if a.library_only else build_all)(force=a.force, ptxas_verbose=a.verbose_ptxas))
