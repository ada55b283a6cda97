"""Builds the gfx950 HIP library (libdg.so) in-tree with hipcc, and the native side of
the Python binding (_binding.so) with g++ where torch and both headers are there.

Usage: python -m moe_grouped_gemm_nt_amd.build [--verbose]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG_DIR, "libdg.so")
CEILINGS_PATH = os.path.join(PKG_DIR, "libdg_ceilings.so")
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")
# source -> extra flags.  The fp32-promotion kernels want MFMA results in
# VGPRs, where the promotion FMAs read them; the power-of-two-scale kernels
# keep their accumulators in AGPRs.
SOURCES = {
    "fp8_gemm.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    "fp8_gemm_e8m0.hip": [],
    "dg_api.hip": [],
    "route.hip": [],
    "expert_rows.hip": [],
    "lora.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    "balance.hip": [],
    "gemv4.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    "grads.hip": [],
}

# packed fp32 VALU forms are disabled on purpose: the kernels issue one fp32
# operation per VALU instruction, the form their results are tested in
HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found; the HIP toolchain (ROCm) is required to build libdg.so")
    return path


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = (r.stdout or "") + (r.stderr or "")
    # the host pass does not know the packed-fp32 feature flag; that warning is expected
    lines = [l for l in out.splitlines() if "packed-fp32-ops" not in l and l.strip()]
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + "\n".join(lines))
    if verbose and lines:
        print("\n".join(lines))


def build(verbose: bool = False, extra_flags=None) -> str:
    objdir = os.path.join(PKG_DIR, "_build")
    os.makedirs(objdir, exist_ok=True)
    jobs = []
    for src, flags in SOURCES.items():
        obj = os.path.join(objdir, src.replace(".hip", ".o"))
        jobs.append(([hipcc()] + HIPCC_FLAGS + flags + list(extra_flags or []) +
                     ["-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj], obj))
    lacks = binding_lacks()
    if os.path.exists(BINDING_PATH):
        os.remove(BINDING_PATH)                    # none of other sources stays beside the library
    # the sources compile independently; one process each
    with ThreadPoolExecutor(max_workers=min(len(jobs) + 1, 8)) as ex:
        binding = None if lacks else ex.submit(build_binding, verbose)
        list(ex.map(lambda j: _run(j[0], verbose), jobs))
    objs = [obj for _, obj in jobs]
    tmp = LIB_PATH + ".tmp"
    _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs, verbose)
    os.replace(tmp, LIB_PATH)
    build_ceilings(verbose)
    if lacks:
        print(f"_binding.so is left out ({lacks}): the calls that it shortens go through ctypes", file=sys.stderr)
    else:
        binding.result()
    return LIB_PATH


def _cxx():
    return shutil.which("g++") or shutil.which("c++")


def binding_lacks() -> str | None:
    """What is missing for _binding.so; libdg.so needs none of it."""
    try:
        import torch
    except ImportError:
        return "torch is not installed"
    if not os.path.exists(os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "autograd",
                                       "python_variable.h")):
        return "torch's headers are not installed"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers are not installed"
    return None if _cxx() else "g++ not found"


def build_binding(verbose: bool = False) -> str:
    """_binding.so: the native side of the Python binding (host code only, against torch's libraries)."""
    lacks = binding_lacks()
    if lacks:
        raise RuntimeError(f"_binding.so cannot be built: {lacks}")
    import torch
    root = os.path.dirname(torch.__file__)
    tmp = BINDING_PATH + ".tmp"
    _run([_cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-isystem", os.path.join(root, "include"),
          "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"), "-o", tmp,
          "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"], verbose)
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def build_ceilings(verbose: bool = False) -> str:
    """libdg_ceilings.so: the MFMA / memory / launch microbenchmarks (include/dg_ceilings.h)."""
    tmp = CEILINGS_PATH + ".tmp"
    _run([hipcc()] + HIPCC_FLAGS + ["-shared", "-I", INCLUDE, os.path.join(CSRC, "ceilings.hip"), "-o", tmp],
         verbose)
    os.replace(tmp, CEILINGS_PATH)
    return CEILINGS_PATH


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
