"""Compile the CUDA library (libsol_attn.so) for sm_100a, in-tree, with nvcc."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libsol_attn.so")
PROFILE_LIB = os.path.join(PKG, "libsol_attn_profile.so")
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_obj")
# Translation units: object name, source, defines.  The norm kernels are compiled once for each pair of types.
_NORMS = (("bf16", "__nv_bfloat16", "__nv_bfloat16"), ("fp16", "__half", "__half"), ("fp32", "float", "float"),
          ("fp32_bf16", "float", "__nv_bfloat16"), ("fp32_fp16", "float", "__half"))
UNITS = [("sol_attn", "sol_attn.cu", ()), ("layer_ops", "layer_ops.cu", ()), ("linear", "linear_launch.cu", ()),
         ("rope", "rope_launch.cu", ())] + [
    (f"norm_{name}", "norm_launch.cu", (f"-DSOLATTN_NORM_NAME=launch_norm_{name}", f"-DSOLATTN_NORM_X={x}",
                                        f"-DSOLATTN_NORM_Y={y}")) for name, x, y in _NORMS]
# What each unit is made of: the attention's headers or the layer operators'.
_COMMON = [os.path.join(CSRC, f) for f in ("host.h", "sm100_ptx.cuh")] + [os.path.join(ROOT, "include", "sol_attn.h")]
_ATTN = [os.path.join(CSRC, f) for f in ("fused.cuh", "moments.cuh", "pool.cuh", "topk_router.cuh")]
_LAYER = [os.path.join(CSRC, f) for f in ("layer_launch.h", "linear.cuh", "norm.cuh", "rope.cuh", "rows.cuh")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libsol_attn.so")


def _deps(source: str):
    return [os.path.join(CSRC, source), *_COMMON, *(_ATTN if source == "sol_attn.cu" else _LAYER)]


def _older(path: str, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(f) > os.path.getmtime(path) for f in deps)


def is_stale(lib: str = LIB) -> bool:
    return _older(lib, {f for _, source, _ in UNITS for f in _deps(source)})


def _run(cmd, verbose: bool):
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr)


def build(force: bool = False, verbose: bool = False, extra_flags=(), profile: bool = False) -> str:
    """Build libsol_attn.so (or, with profile=True, libsol_attn_profile.so with the
    fused kernel's cycle accounting compiled in).  The units are compiled side by
    side; the two libraries share the objects of the layer operators."""
    lib = PROFILE_LIB if profile else LIB
    if not force and not is_stale(lib):
        return lib
    os.makedirs(OBJ, exist_ok=True)
    objects, jobs = [], []
    for name, source, defines in UNITS:
        mine = profile and source == "sol_attn.cu"
        obj = os.path.join(OBJ, f"{name}_profile.o" if mine else f"{name}.o")
        objects.append(obj)
        # the profiling library takes the regular build's objects where they are up to date
        if (force and not (profile and not mine)) or _older(obj, _deps(source)):
            jobs.append([nvcc_path(), "-c", *NVCC_FLAGS, *extra_flags, *defines, *(["-DSOL_ATTN_PROFILE"] if mine else []),
                         "-I", os.path.join(ROOT, "include"), "-o", obj, os.path.join(CSRC, source)])
    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
        list(pool.map(lambda cmd: _run(cmd, verbose), jobs))
    _run([nvcc_path(), *NVCC_FLAGS, "-shared", "-o", lib, *objects], verbose)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, profile="--profile" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
