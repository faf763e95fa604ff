"""Builds the CUDA library in-tree with nvcc for sm_100a.

    python -m exact_attention_117_b200.build [--debug]  (or __graft_entry__.build())

``--debug`` builds ``libfa_b200_debug.so`` with ``-DFA_DEBUG``: the same
kernels with the TMA coordinates, TMEM column ranges and directly indexed
global addresses checked before use (a failed check is reported through the
device error word, see ``fa_check_device_error``).  Point the binding at it
with the ``FA_LIBRARY`` environment variable.  Both also compile
``_fa_binding.so`` (csrc/binding.cpp, host code) with g++ against torch, again when
torch or Python is another one.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfa_b200.so")
BINDING = os.path.join(PKG, "_fa_binding.so")  # Python extension module, host code only
DEBUG_LIB = os.path.join(PKG, "libfa_b200_debug.so")
SOURCES = ["fa_api.cu"]
HEADERS = ["sm100.cuh", "common.cuh", "fwd.cuh", "bwd.cuh", "bwd_main.cuh", "dq_pass.cuh", "kv_outer.cuh",
           "rotary.cuh", "kv4.cuh", "kv4_attend.cuh", "kv4_chunk.cuh", "kv4_host.cuh"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def flags(extra=()):
    return [
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-O3", "-std=c++17", "-lineinfo",
        "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
        "-shared", "--expt-relaxed-constexpr",
        "-I", os.path.join(ROOT, "include"),
        *extra,
    ]


def _stale(lib: str) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "fa.h"))
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def binding_target() -> str:
    """What the extension module is built for, kept beside it in ``_fa_binding.so.for``:
    its code depends on torch's and Python's binary interfaces."""
    import torch
    return f"torch {torch.__version__} {sys.implementation.cache_tag}\n"


def binding_built_for() -> str:
    try:
        with open(BINDING + ".for") as f:
            return f.read()
    except OSError:
        return ""


def _build_binding(force: bool, verbose: bool):
    """csrc/binding.cpp: the Python module between torch tensors and the C ABI."""
    src = os.path.join(CSRC, "binding.cpp")
    deps = [src, os.path.join(ROOT, "include", "fa.h")]
    if not force and os.path.exists(BINDING) and binding_built_for() == binding_target() and \
            all(os.path.getmtime(p) <= os.path.getmtime(BINDING) for p in deps):
        return
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), src, "-o", tmp,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-ltorch_cuda", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    with open(BINDING + ".for", "w") as f:
        f.write(binding_target())


def build(force: bool = False, verbose: bool = False, extra=(), debug: bool = False) -> str:
    lib = DEBUG_LIB if debug else LIB
    _build_binding(force and not debug, verbose)
    if not force and not _stale(lib):
        return lib
    tmp = lib + ".tmp"
    flag_list = flags(list(extra) + (["-DFA_DEBUG"] if debug else []))
    cmd = [nvcc(), *flag_list, "-o", tmp] + [os.path.join(CSRC, s) for s in SOURCES]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
