"""Kernels that start while the kernel before them still runs read what that one writes with ordinary loads: the
non-coherent path (__ldg, and `const ... __restrict__` parameters, which the compiler may send there) is for
data that nothing writes while the grid is resident.  Read from the sources; no GPU."""
import os
import re

import pytest

from paged_kv_cache_175_gb300 import _build


def source(name):
    text = open(os.path.join(_build.CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def kernels(text):
    """(name, parameters, body) of each __global__ function."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s+)?(\w+)\s*\(", text):
        i, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        j = text.index("{", i)
        k, depth = j + 1, 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[k], 0)
            k += 1
        yield m.group(1), text[m.end():i - 1], text[j:k]


@pytest.mark.parametrize("name", ["decode_q8.cu", "decode_mass.cu", "decode_bf16.cu", "decode_tc.cu", "int4.cu", "piece_streams.cuh"])
def test_attention_reads_only_block_tables_past_the_coherent_path(name):
    for arg in re.findall(r"__ldg\(([^;]*)", source(name)):
        assert arg.startswith("a.bt") or (name == "decode_tc.cu" and arg.startswith("row + cur.blk")), arg


# (kernel, parameters that the kernel before it may still be writing)
@pytest.mark.parametrize("name,kernel,written", [("decode_mass.cu", "mass_add_kernel", ["scores", "fin", "mass"]),
                                                 ("cacheblend.cu", "select_top_kernel", ["dev"]), ("cacheblend.cu", "kv_fuse_kernel", ["rows"])])
def test_parameters_written_by_the_kernel_before_are_not_restrict(name, kernel, written):
    found = [p for n, p, body in kernels(source(name)) if n == kernel and "grid_dep_wait" in body]
    assert len(found) == 1
    for w in written:
        assert re.search(r"\*\s*" + w + r"\b", found[0]), (w, found[0])
        assert not re.search(r"__restrict__\s+" + w + r"\b", found[0]), w
