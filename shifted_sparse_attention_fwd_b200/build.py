"""Build the sm_100a shared library (libs2attn.so) in-tree with nvcc, and the torch binding of the serving
entries (_s2torch.so, host code only) with the host compiler.

Usage: python -m shifted_sparse_attention_fwd_b200.build [--verbose]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
SRCS = [os.path.join(PKG_DIR, "csrc", f) for f in ("s2attn_api.cu", "s2serve_api.cu")]
LIB = os.path.join(PKG_DIR, "libs2attn.so")
BINDING_SRC = os.path.join(PKG_DIR, "csrc", "s2_torch.cpp")
BINDING = os.path.join(PKG_DIR, "_s2torch.so")
BINDING_TORCH = os.path.join(PKG_DIR, "_build", "s2torch.version")   # the torch that it was built for
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    csrc = os.path.join(PKG_DIR, "csrc")
    out = [os.path.join(csrc, f) for f in sorted(os.listdir(csrc)) if f.endswith((".cu", ".cuh", ".h"))]
    return out + [os.path.join(ROOT, "include", "s2attn.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def _compile(cmd, out, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose:
        print(res.stdout + res.stderr)
    os.replace(out + ".tmp", out)


def binding_up_to_date() -> bool:
    """Newer than its sources, and built for the torch that is installed."""
    import torch
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_TORCH):
        return False
    with open(BINDING_TORCH) as f:
        built_for = f.read().strip()
    newest = max(os.path.getmtime(f) for f in (BINDING_SRC, os.path.join(ROOT, "include", "s2attn.h")))
    return built_for == torch.__version__ and os.path.getmtime(BINDING) >= newest


def build_binding(verbose: bool = False, force: bool = False) -> str:
    if not force and binding_up_to_date():
        return BINDING
    import torch
    torch_dir = os.path.dirname(torch.__file__)
    inc = os.path.join(torch_dir, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    _compile([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
              "-I", sysconfig.get_paths()["include"], "-I", inc,
              "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda, BINDING_SRC,
              "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
              "-ltorch_python", "-o", BINDING + ".tmp"], BINDING, verbose)
    os.makedirs(os.path.dirname(BINDING_TORCH), exist_ok=True)
    with open(BINDING_TORCH + ".tmp", "w") as f:
        f.write(torch.__version__)
    os.replace(BINDING_TORCH + ".tmp", BINDING_TORCH)
    return BINDING


def build(verbose: bool = False, force: bool = False) -> str:
    """libs2attn.so and the torch binding; returns the library's path."""
    if force or not up_to_date():
        cmd = [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared",
               "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
               "-t", "0",   # the translation units side by side
               "-I", os.path.join(ROOT, "include"), "-o", LIB + ".tmp", *SRCS]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        _compile(cmd, LIB, verbose)
    build_binding(verbose, force)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force=True))
