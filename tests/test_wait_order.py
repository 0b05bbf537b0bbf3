"""Order of a kernel's programmatic-launch controls, read from the sources (no GPU): only behind griddepcontrol.wait
are the results of the kernel before sure to be there."""
import re

import pytest

from test_coherent_loads import kernels, source


@pytest.mark.parametrize("name,kernel,reads", [
    ("decode_q8.cu", "decode_q8_kernel", ["stream_setup(", "produce_streams(", "load_q("]),
    ("decode_mass.cu", "decode_mass_kernel", ["stream_setup(", "produce_streams(", "load_q("]),
    ("decode_mass.cu", "mass_add_kernel", ["clamp_ctx(", "fin[", "mrow[t0"]),
    ("rope_append.cu", "rope_append_kernel", ["a.q ", "a.slots[", "a.positions["]),
    ("q8.cu", "q8_append_kernel", ["a.slots[", "a.tail_seq["]),
    ("evict.cu", "evict_select_kernel", ["a.ctx[", "a.keep[", "a.kept["]),
    ("evict.cu", "evict_move_kernel", ["a.ctx[", "a.counts["])])
def test_serving_kernels_wait_before_they_read(name, kernel, reads):
    body = [b for n, _, b in kernels(source(name)) if n == kernel]
    assert len(body) == 1
    body = body[0]
    wait = body.index("grid_dep_wait();")
    assert not re.search(r"(if|else)\s*(\([^;{]*\))?\s*$", body[:wait])       # unconditional
    assert body[:wait].count("{") - body[:wait].count("}") == 1               # and in no inner block
    for r in reads:
        assert r in body and body.index(r) > wait, r
    if "grid_dep_launch();" in body:                                          # what it lets in finds what it found
        assert body.index("grid_dep_launch();") > wait


def test_a_walk_behind_the_last_sequence_stays_on_it():
    text = source("decode_common.cuh")
    walk = text[text.index("void cursor_next("):]
    walk = walk[:walk.index("template")]
    assert walk.count("min(c.s + 1, a.batch - 1)") == 2 and "++c.s" not in walk


def test_the_merge_reads_lengths_ahead_of_its_wait_from_l2():
    body = [b for n, _, b in kernels(source("decode_plan.cu")) if n == "reduce_kernel"]
    assert len(body) == 1
    early = body[0][:body[0].index("grid_dep_wait();")]
    assert "__ldcg(a.ctx_raw + sq)" in early and "ctx_raw[" not in body[0]
