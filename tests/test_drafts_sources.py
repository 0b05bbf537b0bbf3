"""The kernels of drafted tokens and of the latent cache, read from the sources (no GPU): they start while the kernel before
them still runs, and nothing it may be writing is read before the wait for it, or past the coherent path."""
import ctypes
import re

import pytest

from test_coherent_loads import kernels, source

KERNELS = [("decode_rows.cu", "decode_rows_kernel", ["drafts_of(", "prefetch_l2(", "tma_load", "sh.scan["]),
           ("decode_rows.cu", "rows_join_kernel", ["a.cuts[", "a.ws_ml", "a.ws_o", "tile_of<"]),
           ("latent_append.cu", "latent_append_kernel", ["a.slots[", "a.positions[", "a.kv ", "a.q ", "a.weight"]),
           ("tree_accept.cu", "tree_accept_kernel", ["a.path[", "a.n_accept[", "drafts_of(", "bt["])]


@pytest.mark.parametrize("name,kernel,reads", KERNELS)
def test_kernels_wait_before_they_read(name, kernel, reads):
    body = [b for n, _, b in kernels(source(name)) if n == kernel]
    assert len(body) == 1
    body = body[0]
    wait = body.index("grid_dep_wait();")
    assert not re.search(r"(if|else|for)\s*(\([^;{]*\))?\s*$", body[:wait])
    assert body[:wait].count("{") - body[:wait].count("}") == 1
    for r in reads:
        assert r in body and body.index(r) > wait, r
    assert body.index("grid_dep_launch();") > wait


@pytest.mark.parametrize("name", ["decode_rows.cu", "latent_append.cu", "tree_accept.cu", "drafts.cuh"])
def test_nothing_is_read_past_the_coherent_path(name):
    assert not re.search(r"__ldg|__restrict__|ld\.global\.nc", source(name))


def test_every_wait_ends():
    """Waits on barriers go through the two functions that give up after a limit."""
    text = source("decode_rows.cu")
    assert "mbar_wait(" not in text
    for fn in ("rows_poll", "rows_wait"):
        start = text.index(" " + fn + "(")
        body = text[start:text.index("\n}", start)]
        assert "limit_ns" in body or "rows_poll(bar, round & 1, 2000000000ull" in body
    for m in re.finditer(r"mbar_try_wait\(", text):
        fn = text[:m.start()].rfind("__device__")
        assert re.search(r"rows_(poll|wait)\(", text[fn:m.start()]), text[fn:m.start()][:80]


def test_accept_refuses_caches_that_share_memory():
    """A cache given twice, or two that overlap: rows would move twice.  (Refused before anything is used; no GPU.)"""
    from test_drafts_host import EINVAL, accept
    size = 9 * 2 * 16 * 256                                    # of a cache of the host tests' call
    for ptrs in ((1 << 20, 1 << 20), (1 << 20, (1 << 20) + size - 16), ((1 << 20) + 16, 1 << 20), (1 << 20, 1 << 30, 1 << 20)):
        assert accept(caches=(ctypes.c_void_p * len(ptrs))(*ptrs), n=len(ptrs)) == EINVAL
    assert accept(caches=(ctypes.c_void_p * 2)(1 << 20, (1 << 20) + size), B=0) == 0
