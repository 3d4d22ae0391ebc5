"""Compile libparo.so (the C-ABI library) for gfx950 with hipcc, and _binding.so, in-tree.

Usage: ``python -m rotated_linear_amd._build`` (also called by ``__graft_entry__.build``).
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libparo.so")
ARCH = "gfx950"

COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17", f"-I{INCLUDE}", f"-I{CSRC}",
    # keep packed-FP32 VALU instructions out of the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]
# per-file extras: the build-time pack must round every float64 product and sum on its own
# the GEMM keeps its accumulators in architectural registers (the per-group rescale multiplies them)
EXTRA = {"pack.hip": ["-ffp-contract=off"], "q8_pack.hip": ["-ffp-contract=off"], "gemm.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
         "skinny.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
         # inline assembly names m0, a register the compiler keeps for itself
         "w8a8_column.hip": ["-Wno-inline-asm"], "w8a8_gemm.hip": ["-Wno-inline-asm"]}
SOURCES = ["paro_api.cpp", "schedule.cpp", "pack.hip", "rotate.hip", "decode.hip", "gemm.hip", "skinny.hip", "noalloc.hip",
           "q8_api.cpp", "q8_rows.hip", "q8_rotate.hip", "q8_pack.hip", "w8a8_stream.hip", "w8a8_column.hip", "w8a8_gemm.hip"]


# The 8-bit path's Python calls (binding.cpp): host code only, against torch's headers.
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")


def _hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain is required to build libparo")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src + ".o")
    cmd = [_hipcc(), *COMMON, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_binding() -> bool:
    """The extension saves host time and nothing needs it: without a usable g++ or torch headers the build goes
    on, with a warning, and leaves no older extension behind."""
    torch = importlib.util.find_spec("torch")
    torch_dir = torch.submodule_search_locations[0] if torch else "torch"
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(_hipcc())))
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", f"-I{INCLUDE}",
           f"-I{torch_dir}/include", f"-I{torch_dir}/include/torch/csrc/api/include", f"-I{sysconfig.get_paths()['include']}",
           f"-I{rocm}/include", BINDING_SRC, "-o", tmp, f"-L{torch_dir}/lib", "-lc10", "-lc10_hip", "-ltorch_cpu",
           "-ltorch_python"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}" if r.returncode != 0 else None
    except OSError as e:
        failed = str(e)
    if failed is not None:
        if os.path.exists(BINDING):
            os.remove(BINDING)
        warnings.warn(f"the compiled binding was not built (the 8-bit calls take more host time without it): {failed}", RuntimeWarning)
        return False
    os.replace(tmp, BINDING)
    return True


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
        binding.result()
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
