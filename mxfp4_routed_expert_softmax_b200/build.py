"""Build libk3moe.so in-tree with nvcc for sm_100a, and the Python entry points
of the shortest calls (a module that links torch) with the host compiler.

Run as a script (``python mxfp4_routed_expert_softmax_b200/build.py``): the
package itself refuses to import until the library exists.  With ``--library``,
or without torch, the library alone: nothing but those three Python calls needs
the module."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libk3moe.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
         "-Xcompiler", "-fPIC", "-shared", "-diag-suppress", "177"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def binding_sources():
    return [os.path.join(CSRC, "py_binding.cpp"), os.path.join(INCLUDE, "k3moe.h")]


def torch_version():
    """The installed torch's version (without importing it), or None."""
    from importlib import metadata
    try:
        return metadata.version("torch")
    except metadata.PackageNotFoundError:
        pass
    try:
        import torch
        return torch.__version__
    except ImportError:
        return None


def binding_path():
    """The module's file, or None without torch.  Its name says for which
    interpreter and which torch it is built: under another one it is missing,
    not loaded."""
    version = torch_version()
    return version and os.path.join(PKG, f"_binding-{sys.implementation.cache_tag}-torch{version}.so")


def _older(out: str, srcs) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(s) > os.path.getmtime(out) for s in srcs)


def stale() -> bool:
    binding = binding_path()
    return _older(LIB, sources()) or bool(binding) and _older(binding, binding_sources())


def _compile(cmd, out: str, verbose: bool) -> None:
    tmp = out + f".tmp{os.getpid()}"
    cmd = [*cmd, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, out)


def _binding_command():
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"]]
    for p in include_paths("cuda"):
        cmd += ["-isystem", p]
    return cmd + [binding_sources()[0], "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False, library_only: bool = False) -> str:
    """Compile what is missing or older than its sources."""
    if force or _older(LIB, sources()):
        _compile([NVCC, *FLAGS, "-I", INCLUDE, os.path.join(CSRC, "k3moe_api.cu")], LIB, verbose)
    binding = None if library_only else binding_path()
    if binding and (force or _older(binding, binding_sources())):
        _compile(_binding_command(), binding, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, library_only="--library" in sys.argv))
