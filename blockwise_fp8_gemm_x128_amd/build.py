"""Builds libpuro.so (all HIP kernels + the C ABI) for gfx950 with hipcc, in-tree, and the Python
binding's native half with the host compiler.

Usage: ``python -m blockwise_fp8_gemm_x128_amd.build`` (also called by ``__graft_entry__.build``),
with ``--library`` for the C library alone, which needs neither torch nor a host compiler.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
LIB_PATH = os.path.join(PKG_DIR, "libpuro.so")
SOURCES = ["abi.hip", "quant.hip", "gemm.hip", "optim.hip", "debug.hip", "norm.hip",
           "swiglu.hip", "ckpt.hip", "xent.hip", "ortho.hip"]
# The matrix-core microbenchmark that bench.py --ceiling runs; a library of its own, outside the
# GEMM path.
PROBE_PATH = os.path.join(PKG_DIR, "libpuro_probe.so")
PROBE_SOURCES = ["ceiling.hip"]
# The Python binding's native half: host code against torch's headers.
ARGS_PATH = os.path.join(PKG_DIR, "_args.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    # Packed FP32 ALU ops stay off: every fp32 operation is a plain single-lane instruction.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # Let MFMA results land in VGPRs, where the fp32 promotion reads them directly.
    "-mllvm", "-amdgpu-mfma-vgpr-form=1",
]


def _hipcc(sources, out: str, verbose: bool) -> str:
    srcs = [os.path.join(CSRC, s) for s in sources]
    tmp = out + ".tmp%d" % os.getpid()
    cmd = [HIPCC, *FLAGS, "-I" + INCLUDE, "-I" + CSRC, *srcs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature; that is harmless.
    noise = [l for l in res.stderr.splitlines() if l.strip() and "packed-fp32-ops" not in l]
    if res.returncode != 0:
        sys.stderr.write(res.stderr)
        raise RuntimeError("hipcc failed building " + os.path.basename(out))
    if noise and verbose:
        sys.stderr.write("\n".join(noise) + "\n")
    os.replace(tmp, out)
    return out


def _args(verbose: bool) -> str:
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)), "lib")
    tmp = ARGS_PATH + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           *("-I" + p for p in cpp_extension.include_paths("cpu")),
           "-I" + sysconfig.get_paths()["include"], "-I" + INCLUDE,
           os.path.join(CSRC, "args.cpp"), "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, ARGS_PATH)
    return ARGS_PATH


def build_library(verbose: bool = True) -> str:
    """The C library alone."""
    return _hipcc(SOURCES, LIB_PATH, verbose)


def build(verbose: bool = True) -> str:
    """Everything, the C library first: it is in place also where the binding's half fails."""
    build_library(verbose)
    _hipcc(PROBE_SOURCES, PROBE_PATH, verbose)
    try:
        _args(verbose)
    except (ImportError, OSError, RuntimeError, subprocess.CalledProcessError) as e:
        raise RuntimeError("the binding's native half (%s) failed to build; %s is built" %
                           (os.path.basename(ARGS_PATH), os.path.basename(LIB_PATH))) from e
    return LIB_PATH


if __name__ == "__main__":
    print(build_library() if sys.argv[1:] == ["--library"] else build())
