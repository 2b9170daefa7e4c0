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


def _fresh(path: str, deps, key: str) -> bool:
    """Whether path is at least as new as what it is made of, and was made with these flags (kept beside it)."""
    if not os.path.exists(path) or any(os.path.getmtime(f) > os.path.getmtime(path) for f in deps):
        return False
    try:
        with open(path + ".flags") as f:
            return f.read() == key
    except OSError:
        return False


def _units(extra_flags, profile: bool):
    """(object, source, flags) of each unit."""
    for name, source, defines in UNITS:
        mine = profile and source == "sol_attn.cu"
        yield (os.path.join(OBJ, f"{name}_profile.o" if mine else f"{name}.o"), source,
               [*NVCC_FLAGS, *extra_flags, *defines, *(["-DSOL_ATTN_PROFILE"] if mine else [])])


def _unit_key(source: str, flags) -> str:
    return " ".join([source, *flags])   # no paths: a copy of the tree elsewhere stays fresh


def _lib_key(units) -> str:
    return "\n".join([" ".join([*NVCC_FLAGS, "-shared"]), *(_unit_key(source, flags) for _, source, flags in units)])


def is_stale(lib: str = None, extra_flags=()) -> bool:
    lib = lib or LIB
    units = list(_units(extra_flags, lib == PROFILE_LIB))
    return not _fresh(lib, {f for _, source, _ in units for f in _deps(source)}, _lib_key(units))


def _make(path: str, key: str, flags, inputs, verbose: bool):
    """Compiles into a file of its own, which takes path's place once it is whole."""
    part = f"{path}.{os.getpid()}.part"
    cmd = [nvcc_path(), *flags, "-o", part, *inputs]
    if verbose:
        print(" ".join(cmd))
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
        if os.path.exists(path + ".flags"):
            os.remove(path + ".flags")   # until the new ones stand there, path is not fresh
        os.replace(part, path)
    finally:
        if os.path.exists(part):
            os.remove(part)
    with open(part, "w") as f:
        f.write(key)
    os.replace(part, path + ".flags")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr)


def build(force: bool = False, verbose: bool = False, extra_flags=(), profile: bool = False) -> str:
    """Build libsol_attn.so (or, with profile=True, libsol_attn_profile.so with the
    fused kernel's cycle accounting compiled in).  What is older than its sources, or was
    made with other flags, is compiled, side by side; force compiles all of it, but that
    the profiling library takes the regular one's objects where they are fresh."""
    lib = PROFILE_LIB if profile else LIB
    if not force and not is_stale(lib, extra_flags):
        return lib
    os.makedirs(OBJ, exist_ok=True)
    units = list(_units(extra_flags, profile))
    jobs = []
    for obj, source, flags in units:
        shared = profile and "-DSOL_ATTN_PROFILE" not in flags
        key = _unit_key(source, flags)
        if (force and not shared) or not _fresh(obj, _deps(source), key):
            jobs.append((obj, key, ["-c", *flags, "-I", os.path.join(ROOT, "include")], [os.path.join(CSRC, source)]))
    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
        list(pool.map(lambda job: _make(*job, verbose), jobs))
    _make(lib, _lib_key(units), [*NVCC_FLAGS, "-shared"], [obj for obj, _, _ in units], verbose)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, profile="--profile" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
