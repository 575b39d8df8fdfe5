"""Compile the CUDA library in-tree for sm_100a (nvcc, no JIT cache).

Two builds of the same sources: "release" (lib/libawq_b200.so) and "check"
(lib/libawq_b200_check.so, compiled with -DAWQ_BOUNDS_CHECK: every hand-
addressed global access checks its index and records a failure in a device
word instead of touching memory; see csrc/check.cuh). They need nvcc alone.
Beside them, by g++ against the headers of the installed torch, whose version
is in the name: lib/awq_calls.<python>.torch-<version>.so, the Python module of
csrc/torch_calls.cpp, which holds no kernels and calls whichever build is selected.
"""
from __future__ import annotations

import os
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_DIR = os.path.join(PKG, "lib")
VARIANTS = {
    "release": ("libawq_b200.so", []),
    "check": ("libawq_b200_check.so", ["-DAWQ_BOUNDS_CHECK"]),
}
LIB_PATH = os.path.join(LIB_DIR, VARIANTS["release"][0])
SOURCES = [os.path.join(PKG, "csrc", "awq_lib.cu")]
DEPS = SOURCES + [os.path.join(PKG, "csrc", f) for f in (
    "ptx.cuh", "fq.cuh", "check.cuh", "gemm_sm100.cuh", "gemm_pair_sm100.cuh", "awq_kernels.cuh",
    "w4a16_sm100.cuh", "awq_api.cu", "serve_api.cuh", "w8a8_sm100.cuh", "kv4_sm100.cuh",
    "kv4_prompt_sm100.cuh")] + [os.path.join(ROOT, "include", "awq.h")]

CALLS_DEPS = [os.path.join(PKG, "csrc", "torch_calls.cpp"), os.path.join(ROOT, "include", "awq.h")]

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def lib_path(variant: str = "release") -> str:
    return os.path.join(LIB_DIR, VARIANTS[variant][0])


def torch_version() -> str:
    import importlib.metadata
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return "none"


def calls_path() -> str:
    return os.path.join(LIB_DIR, f"awq_calls.{sys.implementation.cache_tag}.torch-{torch_version()}.so")


def stale(variant: str = "release") -> bool:
    return _older(lib_path(variant), DEPS)


def _older(path, deps) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in deps)


def calls_command(out: str) -> list:
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    if torch.version.cuda is None:
        raise ImportError("torch was built without CUDA")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    include = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"), cuda]
    return ["g++", "-O2", "-std=c++20", "-shared", "-fPIC",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-I" + i for i in include), "-o", out,
            CALLS_DEPS[0], "-L" + os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
            "-ltorch_python"]


def build(force: bool = False, verbose: bool = False, variants=("release",)) -> str:
    """Build the given variants and the calls' module if missing or older than
    their sources (the compilers run for all of them at once). Returns the path
    of the first. Without a CUDA build of torch there is no calls' module."""
    os.makedirs(LIB_DIR, exist_ok=True)
    jobs = []

    def start(path, command):
        cmd = command(path + ".tmp")
        jobs.append((path, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))

    for v in variants:
        if force or stale(v):
            start(lib_path(v), lambda out, v=v: [nvcc(), *NVCC_FLAGS, *VARIANTS[v][1], "-o", out, *SOURCES])
    if force or _older(calls_path(), CALLS_DEPS):
        try:
            start(calls_path(), calls_command)
        except ImportError as e:
            warnings.warn(f"the Python calls' module is not built: {e}")
    failed = []
    for path, cmd, proc in jobs:
        out, _ = proc.communicate()
        if proc.returncode != 0:
            failed.append(os.path.basename(cmd[0]) + " failed:\n" + " ".join(cmd) + "\n" + out)
            continue
        if verbose:
            print(out)
        os.replace(path + ".tmp", path)
    if failed:
        raise RuntimeError("\n".join(failed))
    return lib_path(variants[0])


if __name__ == "__main__":
    print(build(force=True, verbose=True, variants=tuple(VARIANTS)))
