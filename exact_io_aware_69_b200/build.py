"""Build the CUDA libraries libfa.so and libfa_paged.so in-tree (sm_100a only).

``python -m exact_io_aware_69_b200.build`` or ``build_library()``. The CUDA runtime is
linked statically and the driver entry point for TMA descriptors is fetched at run
time, so the library loads on a machine without a GPU (nothing can be launched
there, but every exported symbol can be checked).
"""

from __future__ import annotations

import json
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfa.so")
# ptxas's resource report of the last build (registers and spills per kernel)
RESOURCES = os.path.join(PKG, "libfa.resources.json")
SOURCES = [os.path.join(CSRC, "fa_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")] + [
    os.path.join(INCLUDE, "fa.h")]

# The rotary and paged-cache library: a translation unit of its own that shares
# sm100.cuh and fa_band.cuh with the first.
CSRC_PAGED = os.path.join(PKG, "csrc_paged")
PAGED_LIB = os.path.join(PKG, "libfa_paged.so")
PAGED_RESOURCES = os.path.join(PKG, "libfa_paged.resources.json")
PAGED_SOURCES = [os.path.join(CSRC_PAGED, "fa_paged_api.cu")]
PAGED_DEPS = PAGED_SOURCES + [
    os.path.join(CSRC_PAGED, f) for f in os.listdir(CSRC_PAGED) if f.endswith(".cuh")] + [
    os.path.join(CSRC, f) for f in ("sm100.cuh", "fa_band.cuh")] + [
    os.path.join(INCLUDE, f) for f in ("fa.h", "fa_paged.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "static",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _newer(lib: str, deps) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in deps if os.path.exists(p))


def up_to_date() -> bool:
    return _newer(LIB, DEPS)


def parse_ptxas_report(text: str) -> dict:
    """Registers and spill bytes per kernel from ptxas's -v report: maps each mangled
    kernel name to {"registers", "spill_stores", "spill_loads"}."""
    out, cur = {}, None
    for line in text.splitlines():
        m = re.search(r"Compiling entry function '([^']+)'", line)
        if m:
            cur = m.group(1)
            out[cur] = {"registers": None, "spill_stores": 0, "spill_loads": 0}
            continue
        if cur is None:
            continue
        m = re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", line)
        if m:
            out[cur]["spill_stores"], out[cur]["spill_loads"] = int(m.group(1)), int(m.group(2))
        m = re.search(r"Used (\d+) registers", line)
        if m:
            out[cur]["registers"] = int(m.group(1))
    return out


# Kernels that move registers between warpgroups with setmaxnreg: their split adds up
# to exactly this many registers per thread at launch, so the compiled kernel must use
# exactly that many (the library also refuses to launch otherwise).
FIXED_REGISTERS = {"fa_bwd_main_kernel": 128, "fa_fwd_pp_kernel": 168,
                   "fa_paged_chunk_kernelILi64E": 96, "fa_paged_chunk_kernelILi128E": 168}


def check_resources(report: dict) -> None:
    for name, res in report.items():
        for kernel, regs in FIXED_REGISTERS.items():
            if kernel in name and res["registers"] != regs:
                raise RuntimeError(f"{name}: compiled with {res['registers']} registers per "
                                   f"thread; its register split needs exactly {regs}")


def _compile(lib: str, sources, resources: str, verbose: bool) -> None:
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC, *sources, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose:
        sys.stderr.write(res.stderr)
    report = parse_ptxas_report(res.stderr)
    try:
        check_resources(report)
    except RuntimeError:
        os.unlink(tmp)
        raise
    with open(resources + ".tmp", "w") as fh:
        json.dump(report, fh, indent=1, sort_keys=True)
    os.replace(resources + ".tmp", resources)
    os.replace(tmp, lib)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Build what is out of date (force: everything); returns libfa.so's path."""
    if force or not (up_to_date() and os.path.exists(RESOURCES)):
        _compile(LIB, SOURCES, RESOURCES, verbose)
    if force or not (_newer(PAGED_LIB, PAGED_DEPS) and os.path.exists(PAGED_RESOURCES)):
        _compile(PAGED_LIB, PAGED_SOURCES, PAGED_RESOURCES, verbose)
    return LIB


def resources() -> dict:
    """ptxas's report of the current libfa.so (builds first when it is missing)."""
    build_library()
    with open(RESOURCES) as fh:
        return json.load(fh)


def paged_resources() -> dict:
    """ptxas's report of the current libfa_paged.so."""
    build_library()
    with open(PAGED_RESOURCES) as fh:
        return json.load(fh)


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
