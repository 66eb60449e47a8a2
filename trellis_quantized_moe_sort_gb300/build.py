"""Build libtqmoe.so (the C ABI in include/tqmoe.h) for sm_103a, in-tree.

Compiles each CUDA translation unit with nvcc in parallel and links a shared
library next to this file.  No CMake; about a minute on one core per unit.

    python -m trellis_quantized_moe_sort_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtqmoe.so")
# the binding's short calls (csrc/tq_python.c), by the interpreter that they are built for
CALLS = os.path.join(HERE, "_tqcall" + sysconfig.get_config_var("EXT_SUFFIX"))
CALLS_SOURCES = [os.path.join(CSRC, "tq_python.c"), os.path.join(INCLUDE, "tqmoe.h")]
SOURCES = ["tq_host.cu", "tq_route.cu", "tq_grouped.cu", "tq_gemv.cu", "tq_noalloc.cu", "tq_probe.cu", "tq_mlp.cu", "tq_dequant.cu",
           "tq_router.cu", "tq_fp4_quant.cu", "tq_fp4_gemm.cu", "tq_fp4_gemv.cu", "tq_fp4.cu", "tq_norm.cu", "tq_fp8_quant.cu",
           "tq_fp8_gemm.cu", "tq_few_rows.cu", "tq_fp8.cu", "tq_gemm_f16.cu", "tq_swiglu_linear.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def cuda_home() -> str:
    for cand in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return cand
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    raise RuntimeError("nvcc not found (set CUDA_HOME)")


def python_include() -> str:
    """Folder of Python.h, or an empty string: the binding then calls through ctypes."""
    path = sysconfig.get_paths()["include"]
    return path if os.path.exists(os.path.join(path, "Python.h")) and shutil.which("gcc") else ""


def build_calls(force: bool = False) -> bool:
    """Builds the binding's short calls; False, with none left in place, where that
    cannot be done: the binding then calls through ctypes."""
    include = python_include()
    if include and not force and os.path.exists(CALLS):
        t = os.path.getmtime(CALLS)
        if all(os.path.getmtime(f) <= t for f in CALLS_SOURCES):
            return True
    # one of an earlier source, or without an interpreter's name, must not be imported in its place
    for old in (CALLS, os.path.join(HERE, "_tqcall.so")):
        if os.path.exists(old):
            os.remove(old)
    if not include:
        return False
    tmp = CALLS + ".tmp"
    cmd = ["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I", include, "-I", INCLUDE, CALLS_SOURCES[0], "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(f"calls go through ctypes: gcc failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}\n")
        return False
    os.replace(tmp, CALLS)
    return True


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "tqmoe.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    build_calls(force)
    if not force and up_to_date():
        return LIB
    home = cuda_home()
    nvcc = os.path.join(home, "bin", "nvcc")
    os.makedirs(BUILD, exist_ok=True)
    common = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
                     "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    link = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs + [
        "-Xlinker", f"-rpath,{os.path.join(home, 'lib64')}"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(link)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
