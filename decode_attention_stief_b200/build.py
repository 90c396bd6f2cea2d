"""Build the sm_100a shared library ``libstief.so`` in-tree with nvcc.

Usage: ``python -m decode_attention_stief_b200.build`` (or ``build_library()``).
nvcc cross-compiles for sm_100a without a GPU.  The CUDA runtime is linked
statically so the library loads beside any torch build.

``build_library(variant="testhooks")`` builds ``libstief_testhooks.so`` from the
same sources with ``-DSTIEF_TEST_HOOKS``: bounded waits that give up after 50 ms
and three test-only exports (a setup-barrier stall that makes the waits run out,
a mismatch of a CTA pair's tensor memory, the address of the no-allocation scratch).  Only the timeout tests load it.

``build_marshal()`` builds ``_marshal.so`` with g++: a CPython extension that takes
torch tensors to the library's calls without the cost of doing so in Python.  The
binding works without it, more slowly.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libstief.so")
VARIANTS = {  # name -> (library file, object folder, extra nvcc flags)
    None: ("libstief.so", "_build", []),
    "testhooks": ("libstief_testhooks.so", "_build_testhooks", ["-DSTIEF_TEST_HOOKS"]),
}
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(out: str) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps += glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def library_file(variant=None) -> str:
    return os.path.join(PKG, VARIANTS[variant][0])


def build_library(force: bool = False, verbose: bool = False, extra_flags=(),
                  variant=None) -> str:
    """Compile every csrc/*.cu for sm_100a and link the library next to this file."""
    lib_name, obj_name, variant_flags = VARIANTS[variant]
    lib = os.path.join(PKG, lib_name)
    if not force and not _stale(lib):
        return lib
    extra_flags = [*variant_flags, *extra_flags]
    objdir = os.path.join(PKG, obj_name)
    os.makedirs(objdir, exist_ok=True)
    objs, procs = [], []
    for src in sources():  # the translation units compile side by side
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((cmd, subprocess.Popen(cmd)))
        objs.append(obj)
    failed = [cmd for cmd, proc in procs if proc.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static",
           *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


MARSHAL = os.path.join(PKG, "_marshal.so")


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/marshal.cpp against the running Python and torch."""
    import sysconfig

    import torch
    src = os.path.join(CSRC, "marshal.cpp")
    deps = [src, os.path.join(ROOT, "include", "stief.h"), torch.__file__]
    if not force and os.path.exists(MARSHAL) \
            and all(os.path.getmtime(p) <= os.path.getmtime(MARSHAL) for p in deps):
        return MARSHAL
    home = os.path.dirname(torch.__file__)
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_path("include"),
           "-I", os.path.join(home, "include"), "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           src, "-o", tmp, "-L", os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, MARSHAL)
    return MARSHAL


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True,
                        variant="testhooks" if "--testhooks" in sys.argv else None))
    print(build_marshal(force="--force" in sys.argv, verbose=True))
