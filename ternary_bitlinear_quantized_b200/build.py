"""Build libbitnet_b200.so (nvcc, sm_100a) and the native part of its Python binding (g++) in-tree.

Usage: ``python -m ternary_bitlinear_quantized_b200.build [--verbose]``.  nvcc
cross-compiles without a GPU.  The library links the CUDA runtime statically, so it
does not depend on the runtime version torch ships.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbitnet_b200.so")
BINDING = os.path.join(HERE, "_serving.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh"))]


def build(verbose: bool = False, force: bool = False) -> str:
    hdr = os.path.join(os.path.dirname(HERE), "include", "bitnet_b200.h")
    include = ["-I", os.path.dirname(hdr)]
    _run(LIB, sources() + [hdr], [nvcc(), *ARCH, "-O3", "-std=c++17", "-lineinfo", "--fmad=false", "-Xcompiler", "-fPIC",
                                  "-shared", "-cudart", "static", *include, os.path.join(CSRC, "bitnet_b200.cu"),
                                  *(["-Xptxas=-v"] if verbose else [])], verbose, force)
    src = os.path.join(CSRC, "serving_binding.cpp")
    other = not binding_fits()  # built for another torch or Python
    if force or other or _stale(BINDING, [src, hdr]):
        root = os.path.dirname(torch.__file__)
        cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
        dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], cuda]
        _run(BINDING, [src, hdr], [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                                   f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                                   f'-DSERVING_BUILT_FOR="{built_for()}"',
                                   *[f"-I{d}" for d in dirs], src, "-L" + os.path.join(root, "lib"), "-ltorch_python",
                                   "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-ltorch"], verbose, force or other)
    return LIB


def built_for() -> str:
    """What the native binding depends on beside its source: Python's ABI and torch's."""
    return f"[built for {sysconfig.get_config_var('SOABI')}, torch {torch.__version__}]"


def binding_fits() -> bool:
    """Whether the built binding is there and is for this Python and torch.  The file is read, not loaded: one that does not
    fit may not survive its import."""
    if not os.path.exists(BINDING):
        return False
    with open(BINDING, "rb") as f:
        return built_for().encode() in f.read()


def _stale(out: str, srcs: list[str]) -> bool:
    return not os.path.exists(out) or os.path.getmtime(out) < max(os.path.getmtime(p) for p in srcs + [__file__])


def _run(out: str, srcs: list[str], cmd: list[str], verbose: bool, force: bool) -> None:
    if not force and not _stale(out, srcs):
        return
    cmd = cmd + ["-o", out + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose:
        print(res.stderr, file=sys.stderr)
    os.replace(out + ".tmp", out)


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True)
    print(LIB)
