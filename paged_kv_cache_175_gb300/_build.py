"""In-tree build of libpkv.so for sm_103a (nvcc, translation units compiled in parallel) and of
_calls.so, the binding of its shortest calls (csrc/calls.cpp)."""
from __future__ import annotations

import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpkv.so")
CALLS = os.path.join(PKG, "_calls.so")
SOURCES = ["decode_plan.cu", "decode_bf16.cu", "decode_tc.cu", "int4.cu", "append_rope.cu", "rope_append.cu",
           "q8.cu", "decode_q8.cu", "decode_mass.cu", "evict.cu", "offload.cu", "cacheblend.cu", "probe.cu", "block_manager.cpp"]
HEADERS = ["pkv_device.cuh", "decode_common.cuh", "nvtx_range.h", "umma.cuh", "q8_common.cuh", "piece_streams.cuh", "stream_plan.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def _newest_input() -> float:
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + ["calls.cpp"]] + [
        os.path.join(ROOT, "include", h) for h in ("pkv.h", "pkv_bm.h")] + [__file__]
    return max(os.path.getmtime(p) for p in paths)


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _compile_calls(nvcc: str) -> str:
    obj = os.path.join(OBJ, "calls.o")
    cuda = os.path.dirname(os.path.dirname(nvcc)) if os.path.sep in nvcc else "/usr/local/cuda"
    include = [os.path.join(ROOT, "include"), os.path.join(_torch_dir(), "include"), sysconfig.get_paths()["include"],
               os.path.join(cuda, "include")]
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", *(f"-I{i}" for i in include), "-c",
           os.path.join(CSRC, "calls.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stderr}")
    return obj


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libpkv.so and _calls.so next to this file; returns the library's path."""
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= _newest_input() for p in (LIB, CALLS)):
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose:
            print(r.stderr, end="")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_calls, nvcc)
        objs = list(ex.map(compile_one, SOURCES))
        calls = calls.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    # torch's libraries are in the process when _calls.so is loaded; libpkv.so is found beside it
    tmp = CALLS + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, calls, f"-L{PKG}", "-l:libpkv.so", "-Wl,-rpath,$ORIGIN",
           f"-L{os.path.join(_torch_dir(), 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _calls.so failed:\n{r.stderr}")
    os.replace(tmp, CALLS)
    return LIB


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
