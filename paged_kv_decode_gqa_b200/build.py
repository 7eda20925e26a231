"""Builds the CUDA library and the CPython binding in-tree: paged_kv_decode_gqa_b200/libpagedkv_b200.so
and paged_kv_decode_gqa_b200/_binding.<Python>.torch<version>.so.

    python -m paged_kv_decode_gqa_b200.build [--force] [--verbose-ptxas]

nvcc compiles the single translation unit csrc/pagedkv.cu for sm_100a only,
links the CUDA runtime statically and nothing else (the TMA descriptor entry
point is fetched from the driver at run time). g++ compiles csrc/binding.cpp against the
headers of the PyTorch in use; where there is none, or the compiler fails, the library is
built all the same, and a message says what is missing.
"""
from __future__ import annotations

import glob
import importlib.metadata
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libpagedkv_b200.so")
BINDING_DIR = HERE
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "-shared", "-cudart", "static",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, "pagedkv.h")])


def _older(target, files) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(s) > os.path.getmtime(target) for s in files)


def is_stale() -> bool:
    return _older(LIB, sources())


def binding_path() -> str:
    """The binding of this Python and the PyTorch installed: it belongs to one of each, and its name says which."""
    return os.path.join(BINDING_DIR, f"_binding.{sysconfig.get_config_var('SOABI')}"
                                     f".torch{importlib.metadata.version('torch')}.so")


def build_binding(force: bool = False) -> str:
    """The binding, when it is older than its sources. Raises when it cannot be built."""
    import torch
    binding = binding_path()
    src = os.path.join(CSRC, "binding.cpp")
    if not force and not _older(binding, [src, os.path.join(INCLUDE, "pagedkv.h")]):
        return binding
    from torch.utils import cpp_extension
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = binding + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Wno-attributes",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include")]
    for path in cpp_extension.include_paths():
        cmd += ["-isystem", path]
    cmd += ["-o", tmp, src, "-L", libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, binding)
    return binding


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """The library, which needs nvcc alone, and then the binding, where it can be built."""
    if force or is_stale():
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-o", tmp, os.path.join(CSRC, "pagedkv.cu")]
        if verbose_ptxas:
            cmd[1:1] = ["-Xptxas", "-v"]
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    try:
        build_binding(force)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        print(f"binding not built: {e!r}; only the Python calls of the 8-bit cache, the rotary cache write and the "
              "cache read need it", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv)
    print(LIB)
