"""Build ``libfa_b200.so`` in-tree with nvcc for sm_100a (no JIT, no torch extension).

    python -m io_aware_exact_24_b200.build [--verbose]
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("fa_api.cu", "fa_kv4.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in ("fa_fwd_kernel.cuh", "fa_fwd_persist.cuh", "fa_decode_kernel.cuh", "fa_bwd_kernel.cuh", "sm100_ptx.cuh",
                                                     "exp2_poly.cuh", "fa_kv4_kernel.cuh", "fa_kv4_attend.cuh", "fa_kv4_rows.cuh",
                                                     "fa_internal.h", "fa_kv4_rule.h")] + [
    os.path.join(ROOT, "include", "fa.h")]
OUT = os.path.join(PKG, "libfa_b200.so")
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


# CPython module that marshals the calls of a decoding step (see csrc/fa_fastcall.c)
FAST_SRC = os.path.join(CSRC, "fa_fastcall.c")
FAST_OUT = os.path.join(PKG, "_fastcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def build_fastcall(force: bool = False) -> str:
    """The marshalling module, for this interpreter."""
    if not force and os.path.exists(FAST_OUT) and os.path.getmtime(FAST_SRC) <= os.path.getmtime(FAST_OUT):
        return FAST_OUT
    tmp = FAST_OUT + f".tmp{os.getpid()}"
    subprocess.run([os.environ.get("CC", "gcc"), "-O2", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"],
                    "-o", tmp, FAST_SRC], check=True)
    os.replace(tmp, FAST_OUT)
    return FAST_OUT


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, and the marshalling module, without which only the 4-bit cache calls cannot be made."""
    out = build_library(force, verbose)
    try:
        build_fastcall(force)
    except (OSError, subprocess.CalledProcessError) as e:
        if os.path.exists(FAST_OUT):
            os.remove(FAST_OUT)   # of other sources
        print(f"the 4-bit cache calls are not available from Python: {e}", file=sys.stderr)
    return out


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(OUT):
        t = os.path.getmtime(OUT)
        if all(os.path.getmtime(f) <= t for f in DEPENDS):
            return OUT
    tmp = OUT + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", tmp,
           *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
