"""Compile the CUDA library libattn_b200.so in-tree for sm_100a, and the Python
binding attn_bind.so of its entry points for paged caches (that only where torch
is installed).

Usage: python -m exact_softmax_attention_04_b200.build_lib [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import importlib.metadata
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libattn_b200.so")
BIND = os.path.join(PKG, "attn_bind.so")
BIND_SOURCE = os.path.join(CSRC, "bind.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("attn_api.cu", "attn_bwd_api.cu", "attn_decode_api.cu",
                                             "attn_paged_api.cu", "attn_pages_api.cu")]
HEADERS = [os.path.join(CSRC, f) for f in ("attn_fwd_kernel.cuh", "attn_bwd_kernel.cuh",
                                            "attn_bwd_fused_kernel.cuh", "attn_decode_kernel.cuh",
                                            "attn_paged_plan.cuh", "attn_paged_kernel.cuh",
                                            "attn_latent_kernel.cuh", "attn_pages_kernel.cuh", "sm100.cuh",
                                            "attn_host.h")] + [
    os.path.join(ROOT, "include", "attn.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "-shared",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in SOURCES + HEADERS)


def torch_version():
    """Of the torch that is installed, or None. (The C library needs none.)"""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def bind_record() -> str:
    """The file that says what the binding was built for."""
    return os.path.join(os.path.dirname(BIND), "_build", "attn_bind.txt")


def bind_for() -> str:
    return f"torch {torch_version()}, {sysconfig.get_config_var('SOABI')}"


def bind_stale() -> bool:
    if not os.path.exists(BIND) or not os.path.exists(bind_record()):
        return True
    with open(bind_record()) as f:
        if f.read() != bind_for():
            return True
    t = os.path.getmtime(BIND)
    return any(os.path.getmtime(f) > t for f in (BIND_SOURCE, os.path.join(ROOT, "include", "attn.h")))


def build_bind() -> str:
    """attn_bind.so, next to the library and against it and torch's."""
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-o", tmp, BIND_SOURCE, "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
           "-ltorch", "-lc10_cuda", "-lc10", "-L", PKG, "-l:libattn_b200.so", "-Wl,-rpath,$ORIGIN"]
    subprocess.check_call(cmd)
    os.replace(tmp, BIND)
    os.makedirs(os.path.dirname(bind_record()), exist_ok=True)
    with open(bind_record(), "w") as f:
        f.write(bind_for())
    return BIND


def build(force: bool = False, verbose: bool = False) -> str:
    if force or stale():
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc()] + NVCC_FLAGS + ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        cmd += ["-o", tmp] + SOURCES
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    if force or bind_stale():
        if torch_version() is None:
            print(f"torch is not installed: {os.path.basename(BIND)}, the binding for it, is not built", file=sys.stderr)
        else:
            build_bind()
    return LIB


def build_variant(out_path: str, defines) -> str:
    """Build the same sources with extra preprocessor definitions into
    ``out_path`` (used by the fault-injection test; never the library)."""
    cmd = [_nvcc()] + NVCC_FLAGS + ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    cmd += [f"-D{d}" for d in defines]
    cmd += ["-o", str(out_path)] + SOURCES
    subprocess.check_call(cmd)
    return str(out_path)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force or a.verbose, verbose=a.verbose), file=sys.stderr)
