"""Builds libdense_gemm_tn.so in-tree with nvcc for sm_103a (no torch
extension machinery: the library is a plain C-ABI shared object), and the
CPython-API binding of its compute calls (_tn_fast, gcc) where the Python
headers are installed."""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdense_gemm_tn.so")
SOURCES = [os.path.join(CSRC, f) for f in ("tn_gemm.cu", "layers.cu", "w4.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in ("tn_gemm_kernel.cuh", "sm103_ptx.cuh", "quant_e4m3_kernel.cuh", "repack_kernel.cuh",
                                                     "aux_kernels.cuh", "skinny_kernel.cuh", "grouped_kernel.cuh", "grouped_ptx.cuh", "grouped_host.cuh", "grouped_calls.cuh", "host_common.cuh", "i8_kernel.cuh",
                                                     "quant_i8_kernel.cuh", "grouped_sinks.cuh", "sinks_host.cuh",
                                                     "w4_kernel.cuh", "w4_host.cuh", "gated_few_kernel.cuh", "layers_kernels.cuh")] + [
    os.path.join(INCLUDE, "tn_gemm.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


OBJECTS = os.path.join(PKG, "build")


def object_path(source: str) -> str:
    return os.path.join(OBJECTS, os.path.splitext(os.path.basename(source))[0] + ".o")


def compile_cmds(verbose_ptxas: bool = False) -> list[list[str]]:
    """One command per translation unit, to be run side by side (the three take about
    as long each; nvcc's own --split-compile is not used: it cost the kernels 10 to 80 %)."""
    os.makedirs(OBJECTS, exist_ok=True)
    flags = ["-std=c++17", "-O3", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-diag-suppress", "1160", "-I", INCLUDE]
    if verbose_ptxas:
        flags.insert(0, "-Xptxas=-v")
    return [[nvcc(), *flags, "-c", "-o", object_path(s), s] for s in SOURCES]


def link_cmd() -> list[str]:
    return [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", LIB, *map(object_path, SOURCES)]


def run_all(cmds: list[list[str]]) -> None:
    """Runs the commands side by side."""
    procs = [subprocess.Popen(c) for c in cmds]
    for cmd, rc in zip(cmds, [p.wait() for p in procs]):
        if rc != 0:
            raise RuntimeError(f"build step failed ({rc}): {' '.join(cmd)}")


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in DEPENDS)


def build(force: bool = False) -> str:
    if force or stale():
        run_all(compile_cmds())
        subprocess.check_call(link_cmd())
    return LIB


FAST_SRC = os.path.join(CSRC, "pyfast.c")
FAST = os.path.join(PKG, "_tn_fast" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


def fast_build_cmd() -> list[str] | None:
    """gcc command for the CPython-API binding, or None without Python.h.  It
    links libdense_gemm_tn.so by an $ORIGIN run path, so the process shares the
    one copy of the library that the ctypes binding loads."""
    inc = sysconfig.get_paths().get("include", "")
    if not inc or not os.path.exists(os.path.join(inc, "Python.h")):
        return None
    cc = shutil.which("gcc") or shutil.which("cc") or "gcc"
    return [cc, "-O2", "-std=c11", "-shared", "-fPIC", "-Wall", "-I", INCLUDE, "-I", inc, "-o", FAST, FAST_SRC,
            "-L", PKG, "-ldense_gemm_tn", "-Wl,-rpath,$ORIGIN"]


def fast_stale() -> bool:
    if not os.path.exists(FAST):
        return True
    t = os.path.getmtime(FAST)
    return any(os.path.getmtime(f) > t for f in (FAST_SRC, os.path.join(INCLUDE, "tn_gemm.h"), LIB))


def build_fast(force: bool = False) -> str | None:
    """Builds the binding after the library; returns its path, or None when the
    Python headers are missing (the ctypes binding of the same calls remains)."""
    cmd = fast_build_cmd()
    if cmd is None:
        return None
    if force or fast_stale():
        subprocess.check_call(cmd)
    return FAST
