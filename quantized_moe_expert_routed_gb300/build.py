"""Build libmnw_moe.so in-tree with nvcc for sm_103a.

Each translation unit compiles in parallel, then one nvcc link makes the
shared library next to this file.  The binding of the decode step's calls
(csrc/mnw_calls.cpp, a Python module on torch's C++ interface) compiles beside
them with the host compiler; where it cannot, the library is built all the
same, and those calls go through their Python form.  No CMake, no torch
extension machinery.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmnw_moe.so")
SOURCES = ["mnw_api.cu", "mnw_route.cu", "mnw_router.cu", "mnw_quant.cu", "mnw_gemm.cu", "mnw_gemm_rows.cu", "mnw_gemm_rows_a8.cu", "mnw_gemm_warp.cu",
           "mnw_gemm_warp_dep.cu", "mnw_static_ws.cu", "mnw_selftest.cu", "mnw_attention.cu",
           "mnw_norm.cu", "mnw_kv_append.cu", "mnw_attn_paged.cu",
           "mnw_attn_paged_block.cu", "mnw_attn_paged_int4.cu", "mnw_kv_values.cu", "mnw_lora.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2", "-Xcompiler", "-fvisibility=hidden",
         "-I", CSRC, "-I", INCLUDE]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libmnw_moe.so")
    return cand


def calls_path() -> str:
    """The binding's file, for one torch and one Python, whose C++ interfaces differ between versions."""
    import torch
    return os.path.join(HERE, "mnw_calls_" + re.sub(r"\W", "_", torch.__version__) + sysconfig.get_config_var("EXT_SUFFIX"))


def calls_failed() -> str:
    """Where the reason stands that the binding could not be compiled; a source newer than it is tried again."""
    return calls_path() + ".failed.txt"


def _compile_calls() -> None:
    calls = calls_path()
    tmp = calls + f".{os.getpid()}.tmp"
    try:
        import torch
        root = os.path.dirname(torch.__file__)
        include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                   sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"), INCLUDE]
        lib = os.path.join(root, "lib")
        cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *(f for i in include for f in ("-isystem", i)),
               os.path.join(CSRC, "mnw_calls.cpp"), "-o", tmp, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu",
               "-ltorch_python", f"-Wl,-rpath,{lib}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = None if r.returncode == 0 else f"the compiler failed on mnw_calls.cpp:\n{r.stderr}"
    except (OSError, RuntimeError) as e:  # no compiler
        why = f"mnw_calls.cpp was not compiled: {e}"
    if why is None:
        os.replace(tmp, calls)
        return
    if os.path.exists(calls):  # of older sources
        os.remove(calls)
    with open(tmp, "w") as f:
        f.write(why)
    os.replace(tmp, calls_failed())


def _deps():
    # sources, the public header and this file (its flags)
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "mnw_moe.h"),
                                                                 os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False) -> str:
    new = _deps()
    fresh = lambda f: not force and os.path.exists(f) and os.path.getmtime(f) >= new  # noqa: E731
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = None if fresh(calls_path()) or fresh(calls_failed()) else ex.submit(_compile_calls)
        if not fresh(LIB):
            _build_library(ex, verbose)
        if calls:
            calls.result()
    return LIB


def _build_library(ex, verbose: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".{os.getpid()}.tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
