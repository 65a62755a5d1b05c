"""Build the sm_100a CUDA library ``libmoe_b200.so`` in-tree with nvcc, and ``_binding`` (its dense
operators on torch tensors) with g++ and torch's headers.  Where those are missing the library is built all the
same, with a warning: everything but the dense operators works without ``_binding``.

    python -m sparse_moe_rmsnorm_b200.build [--force] [--verbose]

The library links the CUDA runtime statically and reaches the driver's
tensor-map encoder through ``cudaGetDriverEntryPoint``, so it loads (and its
symbols can be inspected) on a machine without a GPU driver.
"""
from __future__ import annotations

import argparse
import glob
import importlib.metadata
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe_b200.so")
HEADER = os.path.join(ROOT, "include", "moe_b200.h")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [HEADER, __file__]
    return any(os.path.getmtime(p) > t for p in deps)


def _binding_stale(built_for: str) -> bool:
    """Whether ``_binding`` is missing, older than its sources, or built for another torch than installed."""
    if not os.path.exists(BINDING):
        return True
    t = os.path.getmtime(BINDING)
    if any(os.path.getmtime(p) > t for p in (BINDING_SRC, HEADER, __file__)):
        return True
    with open(BINDING, "rb") as f:
        return built_for.encode() + b"\0" not in f.read()


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The torch extension over the library (which it links, and has to be there).  Raises where it cannot be built."""
    built_for = "moe_b200 binding for torch " + importlib.metadata.version("torch")
    if not force and not _binding_stale(built_for):
        return BINDING
    import torch
    from torch.utils import cpp_extension

    tmp = BINDING + ".tmp.%d" % os.getpid()
    includes = [os.path.dirname(HEADER), sysconfig.get_paths()["include"],
                *cpp_extension.include_paths(device_type="cuda")]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           '-DMOE_BINDING_BUILT_FOR="%s"' % built_for,
           *[f for d in includes for f in ("-isystem", d)], "-o", tmp, BINDING_SRC,
           "-L" + HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           *["-L" + d for d in cpp_extension.library_paths(device_type="cuda")],
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, nvcc: str = "nvcc") -> str:
    if force or _stale():
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.dirname(HEADER), "-shared", "-Xlinker",
               "-soname=" + os.path.basename(LIB), "-o", tmp, *sources(), "-cudart", "static"]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    try:
        build_binding(force, verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:     # (no torch, no g++, no headers)
        warnings.warn("libmoe_b200.so is built, but not the torch binding of the dense 8-bit operators, which needs "
                      "torch with its headers and g++: %s: %s" % (type(e).__name__, e))
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
