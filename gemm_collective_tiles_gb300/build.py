"""Build the in-tree shared library ``_lib/libgemm_collective_tiles.so`` with
nvcc for sm_103a (five translation units, compiled side by side; no PyTorch
headers involved).

Usage: ``python -m gemm_collective_tiles_gb300.build`` or ``build()``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_FP8 = os.path.join(PKG, "csrc_fp8")
CSRC_BLOCK = os.path.join(PKG, "csrc_block")
LIBDIR = os.path.join(PKG, "_lib")
LIBNAME = "libgemm_collective_tiles.so"
SOURCES = [os.path.join(CSRC, "iris_api.cu"), os.path.join(CSRC_FP8, "fp8_api.cu"),
           *(os.path.join(CSRC_BLOCK, f) for f in ("block_api.cu", "norm_api.cu", "norm_grad_api.cu", "norm_grad_post.cu"))]
HEADERS = [os.path.join(CSRC, f) for f in ("fused_kernel.cuh", "ptx.cuh")]
HEADERS += [os.path.join(CSRC_FP8, f) for f in ("fp8_ptx.cuh", "fp8_elem.cuh", "fp8_wait.cuh", "fp8_repack.cuh", "fp8_quant.cuh",
                                                "fp8_gemm.cuh", "fp8_few.cuh", "fp8_host.cuh")]
HEADERS += [os.path.join(CSRC_BLOCK, f) for f in ("act.cuh", "block_gemm.cuh", "block_few.cuh", "block_elem.cuh",
                                                  "block_norm.cuh", "block_host.cuh", "norm_host.cuh", "norm_grad.cuh")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def lib_path() -> str:
    return os.path.join(LIBDIR, LIBNAME)


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = SOURCES + HEADERS
    deps.append(os.path.join(ROOT, "include", "gemm_collective_tiles.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile the library if any source is newer than it; return its path."""
    out = lib_path()
    if not force and not _stale(out):
        return out
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = out + f".{os.getpid()}.tmp"
    cmd = [nvcc_path(), "-O3", "-std=c++17", "-lineinfo", *ARCH,
           "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-DGCT_BUILD", "--threads", str(len(SOURCES)), "-o", tmp]
    if extra_flags:
        cmd += list(extra_flags)
    cmd += SOURCES
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, file=sys.stderr)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
