"""In-tree build of libpkv.so for sm_103a (nvcc, translation units compiled in parallel) and of
_calls.so, the binding of its shortest calls (csrc/calls.cpp)."""
from __future__ import annotations

import os
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpkv.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_KEY = os.path.join(OBJ, "calls.key")             # what CALLS was built for
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


def _newest(*names: str) -> float:
    paths = [os.path.join(CSRC, f) for f in names] + [
        os.path.join(ROOT, "include", h) for h in ("pkv.h", "pkv_bm.h")] + [__file__]
    return max(os.path.getmtime(p) for p in paths)


def _run(what: str, cmd: list[str]) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")
    return r.stderr


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def calls_key() -> str:
    """What _calls.so is bound to besides its source: the C++ interface of one torch, and one Python's."""
    import torch
    return f"{torch.__version__} {_torch_dir()} {sysconfig.get_config_var('EXT_SUFFIX')}"


def calls_current() -> bool:
    """Whether _calls.so is there and was built for this torch and this Python."""
    try:
        with open(CALLS_KEY) as f:
            return os.path.exists(CALLS) and f.read() == calls_key()
    except OSError:
        return False


def _compile_calls(nvcc: str) -> str:
    obj = os.path.join(OBJ, "calls.o")
    cuda = os.path.dirname(os.path.dirname(nvcc)) if os.path.sep in nvcc else "/usr/local/cuda"
    include = [os.path.join(ROOT, "include"), os.path.join(_torch_dir(), "include"), sysconfig.get_paths()["include"],
               os.path.join(cuda, "include")]
    _run("g++ on calls.cpp", ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", *(f"-I{i}" for i in include), "-c",
                              os.path.join(CSRC, "calls.cpp"), "-o", obj])
    return obj


def _link_calls(obj: str) -> None:
    # torch's libraries are in the process when _calls.so is loaded; libpkv.so is found beside it
    tmp = CALLS + ".tmp"
    _run("link of _calls.so", ["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libpkv.so", "-Wl,-rpath,$ORIGIN",
                               f"-L{os.path.join(_torch_dir(), 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, CALLS)
    with open(CALLS_KEY, "w") as f:
        f.write(calls_key())


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libpkv.so next to this file, and _calls.so behind it; returns the library's path.  The
    library needs neither Python nor torch: where _calls.so cannot be built it is there all the same, with a
    warning, and the calls that go through _calls.so refuse to run."""
    def fresh(path, *names):
        return not force and os.path.exists(path) and os.path.getmtime(path) >= _newest(*names)

    lib_fresh = fresh(LIB, *SOURCES, *HEADERS)
    calls_fresh = fresh(CALLS, "calls.cpp") and calls_current()
    if lib_fresh and calls_fresh:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
        out = _run(f"nvcc on {src}", [nvcc, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])
        if verbose:
            print(out, end="")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = None if calls_fresh else ex.submit(_compile_calls, nvcc)
        if not lib_fresh:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + ".tmp"
            _run("link", [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-ldl"])
            os.replace(tmp, LIB)
        if calls is not None:
            try:
                _link_calls(calls.result())
            except (RuntimeError, OSError, ImportError) as e:
                warnings.warn(f"_calls.so was not built: {e}", stacklevel=2)
    return LIB


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
