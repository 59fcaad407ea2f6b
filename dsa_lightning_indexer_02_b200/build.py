"""Build libdsa.so (sm_100a) in-tree with nvcc, and with the host compiler the binding's marshalling module, which
links it.  No GPU is needed to build.

build_lib() makes the library alone, for C callers: nvcc is all it needs.  build() adds the module, which needs the
headers of the running interpreter and of torch; without it the binding makes its calls through ctypes, slower by
some 10 us each.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "dsa_lib.cu")
LIB = os.path.join(HERE, "libdsa.so")
DEPS = [os.path.join(HERE, "csrc", f) for f in (
    "dsa_lib.cu", "ptx.cuh", "indexer.cuh", "topk.cuh", "attn.cuh", "attn_dedup.cuh", "kl.cuh", "rope.cuh",
    "kv8.cuh", "paged_attn.cuh")]
DEPS += [os.path.join(ROOT, "include", "dsa.h"), os.path.abspath(__file__)]

MARSHAL_SRC = os.path.join(HERE, "csrc", "marshal.cpp")

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "-Xptxas", "-v", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in DEPS)


def marshal_path() -> str:
    """Where the marshalling module for the running interpreter and torch lies.  It is compiled against the inline
    code of both, so its name holds what must agree: a module of others is never loaded, and theirs is built anew."""
    import sysconfig
    import torch
    abi = f"{sysconfig.get_config_var('SOABI')}-torch-{torch.__version__}-{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(HERE, f"_marshal.{abi}.so")


def build_marshal(force: bool = False) -> str | None:
    """The marshalling module; None, with a message, where torch or the host compiler is missing."""
    try:
        import torch
        out = marshal_path()
    except ImportError as e:
        sys.stderr.write(f"marshalling module not built: {e}\n")
        return None
    deps = (MARSHAL_SRC, os.path.join(ROOT, "include", "dsa.h"), os.path.abspath(__file__))
    if not force and os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps):
        return out
    import sysconfig
    top = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"], "-isystem", f"{top}/include",
           "-isystem", f"{top}/include/torch/csrc/api/include", "-isystem", f"{cuda}/include", MARSHAL_SRC,
           "-o", out + ".tmp", LIB, f"-L{top}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{top}/lib"]
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
    except FileNotFoundError as e:
        sys.stderr.write(f"marshalling module not built: {e}\n")
        return None
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("the host compiler failed building the marshalling module")
    os.replace(out + ".tmp", out)
    return out


def build(force: bool = False, verbose: bool = False) -> str:
    """The library and the marshalling module."""
    lib = build_lib(force, verbose)
    build_marshal(force)
    return lib


def build_lib(force: bool = False, verbose: bool = False) -> str:
    """libdsa.so alone, whose interface is include/dsa.h."""
    if not force and up_to_date():
        return LIB
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), SRC, "-Xlinker", "-soname=libdsa.so", "-o", LIB + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libdsa.so")
    with open(os.path.join(HERE, "ptxas_info.txt"), "w") as f:
        f.write(res.stderr)
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    (build_lib if "--lib" in sys.argv else build)(force="--force" in sys.argv, verbose=True)
    print(LIB)
