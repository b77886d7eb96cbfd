"""Build libfathom.so in-tree for sm_100a with nvcc, and _binding.so with g++.

Each translation unit is compiled to an object under _build/ (in parallel),
then linked into decode_fathom_plan_b200/libfathom.so.  _binding.so is the
Python module that passes torch tensors to the library's calls on a paged
cache (csrc/binding.cpp).  Each is rebuilt only when a source or header is
newer than it, the module also when torch is another than it was built for.
The library needs neither torch nor its headers: where they are missing it is
built alone, and the calls that take tensors of a paged cache raise.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfathom.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfathom.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def torch_mark() -> bytes:
    """What _binding.so holds of the torch that it was built for (empty: none here)."""
    from importlib import metadata
    try:
        return ("built for torch " + metadata.version("torch") + ";").encode()
    except metadata.PackageNotFoundError:
        return b""


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING):
        return False
    t = os.path.getmtime(BINDING)
    with open(BINDING, "rb") as f:
        if torch_mark() not in f.read():
            return False
    return all(os.path.getmtime(p) <= t for p in
               [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))


def binding_lacks() -> str:
    """What this machine lacks to build _binding.so; empty where it has all."""
    import sysconfig
    if not torch_mark():
        return "torch is not installed"
    from torch.utils import cpp_extension
    dirs = cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]
    for header in ("torch/csrc/autograd/python_variable.h", "Python.h"):
        if not any(os.path.exists(os.path.join(d, header)) for d in dirs):
            return header + " is missing"
    if not shutil.which(cxx()):
        return cxx() + " is missing"
    return ""


def cxx() -> str:
    return os.environ.get("CXX") or "g++"


def build_binding(verbose: bool = False):
    """Compile _binding.so against torch's headers and libfathom.so (beside it)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include")] + \
        cpp_extension.include_paths()
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [cxx(), "-O2", "-std=c++17", "-fPIC",
           "-shared", '-DFATHOM_TORCH_MARK="%s"' % torch_mark().decode(), "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI] + \
        [x for i in includes for x in ("-isystem", i)] + [BINDING_SRC, "-o", tmp, "-L" + PKG,
         "-l:libfathom.so", "-L" + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
         "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    if verbose:
        print(" ".join(cmd))
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if p.returncode != 0:
        raise RuntimeError("g++ failed:\n" + p.stdout.decode(errors="replace"))
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    build_library(force, verbose, ptxas_info)
    if force or not binding_up_to_date():
        lacks = binding_lacks()
        if lacks:
            if os.path.exists(BINDING):          # of another source or torch: not to be loaded
                os.remove(BINDING)
            print(f"{BINDING} is not built: {lacks}", file=sys.stderr)
        else:
            build_binding(verbose)
    return LIB


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [cc] + ARCH + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + \
            ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose or ptxas_info:
            sys.stdout.write(text)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError("nvcc failed:\n" + msg)
    tmp = LIB + ".tmp%d" % os.getpid()
    link = [cc] + ARCH + ["-shared", "-o", tmp] + objs
    if verbose:
        print(" ".join(link))
    subprocess.check_call(link)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv,
          ptxas_info="--ptxas" in sys.argv)
    print(LIB)
