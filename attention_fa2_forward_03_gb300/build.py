"""Builds the CUDA library in-tree with nvcc (sm_103a only).

    python -m attention_fa2_forward_03_gb300.build
"""
from __future__ import annotations

import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfa2.so")
# The same sources with FA2_DEBUG: device-side bounds checks that report
# FA2_ERR_BOUNDS instead of touching memory outside the planned extents.
DEBUG_LIB = os.path.join(PKG, "libfa2_debug.so")
SOURCES = [os.path.join(CSRC, "fa2_fwd_sm103.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, "ptx_sm103.cuh"), os.path.join(CSRC, "fa2_fwd_sm103.cuh"), os.path.join(CSRC, "fa2_bwd_sm103.cuh"), os.path.join(CSRC, "fa2_fwd_fp8_sm103.cuh"),
                     os.path.join(CSRC, "fa2_fwd_d64_sm103.cuh"), os.path.join(CSRC, "fa2_kv4_sm103.cuh"),
                     os.path.join(CSRC, "fa2_kv4_tc_sm103.cuh"),
                     os.path.join(INCLUDE, "fa2.h")]
# The extension that passes torch tensors to the KV cache entry points (host code only), and the torch it was built for.
TORCH_LIB = os.path.join(PKG, "_kv4_torch.so")
TORCH_STAMP = TORCH_LIB + ".for"
TORCH_SOURCES = [os.path.join(CSRC, "kv4_torch.cpp")]
TORCH_DEPENDS = TORCH_SOURCES + [os.path.join(INCLUDE, "fa2.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def installed_torch():
    """(version, folder) of the torch that the extension is built against,
    found without importing it; None without torch or its headers."""
    try:
        spec = importlib.util.find_spec("torch")
    except ValueError:
        spec = None
    if spec is None or not spec.origin:
        return None
    root = os.path.dirname(spec.origin)
    if not os.path.exists(os.path.join(root, "include", "torch", "csrc", "autograd", "python_variable.h")):
        return None
    return str(runpy.run_path(os.path.join(root, "version.py"))["__version__"]), root


def built_for():
    """Version of the torch that the extension was built for; None if there is none."""
    try:
        with open(TORCH_STAMP) as f:
            return f.read().strip()
    except OSError:
        return None


def needs_build(lib: str = LIB) -> bool:
    if lib == TORCH_LIB:
        torch = installed_torch()
        if torch is None:
            return False
        if torch[0] != built_for():
            return True
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in (TORCH_DEPENDS if lib == TORCH_LIB else DEPENDS))


def torch_command(out: str, root: str) -> list:
    """g++ command of the extension, against the torch in `root`."""
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, "-I", os.path.join(root, "include"), "-I",
            os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"), "-I",
            sysconfig.get_paths()["include"], "-o", out, *TORCH_SOURCES, "-L", os.path.join(root, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libfa2.so, libfa2_debug.so and the torch extension next to this
    file (in parallel) if they are missing or stale; returns the release
    library's path. The C libraries need nvcc alone: without torch there is no
    extension, and one that does not compile leaves them in place."""
    jobs = []
    for lib, extra in ((LIB, []), (DEBUG_LIB, ["-DFA2_DEBUG"])):
        if not force and not needs_build(lib):
            continue
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
               *extra, "-I", INCLUDE, "-o", tmp, *SOURCES]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        jobs.append((subprocess.Popen(cmd), tmp, lib, cmd))
    torch = installed_torch()
    if torch is not None and (force or needs_build(TORCH_LIB)):
        tmp = TORCH_LIB + f".tmp{os.getpid()}"
        cmd = torch_command(tmp, torch[1])
        jobs.append((subprocess.Popen(cmd), tmp, TORCH_LIB, cmd))
    failed = None
    for proc, tmp, lib, cmd in jobs:
        if proc.wait() != 0:
            failed = failed or subprocess.CalledProcessError(proc.returncode, cmd)
            continue
        os.replace(tmp, lib)
        if lib == TORCH_LIB:
            with open(TORCH_STAMP, "w") as f:
                f.write(torch[0] + "\n")
    if failed:
        raise failed
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
