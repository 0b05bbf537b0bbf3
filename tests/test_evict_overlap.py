"""kv_evict's outputs that lie over one another, or over what is still read, are refused before anything is launched.
Host memory stands for the tensors; no GPU."""
import ctypes

import pytest

import paged_kv_cache_175_gb300 as pkv
from paged_kv_cache_175_gb300 import _build

BATCH, N_KV, STRIDE = 4, 2, 40


@pytest.fixture(scope="module")
def call():
    _build.build_library()
    L = pkv.lib()
    buf = (ctypes.c_uint8 * (1 << 20))()
    base = (ctypes.addressof(buf) + 255) & ~255
    at = {n: base + 16384 * i for i, n in enumerate("ctx keep mass pos kept dropped mass_out pos_out kept_out dropped_out new pool ws".split())}

    def evict(in_place=False, stream=None, **k):
        a = dict(at, **k)
        if in_place:
            a.update(mass_out=a["mass"], pos_out=a["pos"], kept_out=a["kept"], dropped_out=a["dropped"])
        return L.pkv_kv_evict(a["pool"], a["pool"], a["ctx"], 2, a["ctx"], a["keep"], 0, a["mass"], a["pos"], a["kept"], a["dropped"], a["mass_out"],
                              a["pos_out"], a["kept_out"], a["dropped_out"], STRIDE, a["new"], BATCH, N_KV, 64, 16, 4, a["ws"], 1 << 16, None, stream)
    evict.at, evict.buf = at, buf
    return evict


@pytest.mark.parametrize("first,second", [("new", "kept_out"), ("new", "dropped_out"), ("kept_out", "dropped_out"), ("kept_out", "ctx"), ("kept_out", "keep"),
                                          ("kept_out", "kept"), ("kept_out", "dropped"), ("dropped_out", "ctx"), ("dropped_out", "keep"),
                                          ("dropped_out", "kept"), ("dropped_out", "dropped"), ("new", "ctx"), ("new", "keep"), ("new", "kept"), ("new", "dropped")])
def test_lengths_and_counts(call, first, second):
    for shift in (-4 * (BATCH - 1), -4, 0, 4, 4 * (BATCH - 1)):
        assert call(**{first: call.at[second] + shift}) == -1, shift


@pytest.mark.parametrize("first,second", [("mass_out", "pos_out"), ("mass_out", "mass"), ("mass_out", "pos"), ("pos_out", "mass"), ("pos_out", "pos")])
def test_rows(call, first, second):
    rows = 4 * ((BATCH * N_KV - 1) * STRIDE + 32)
    for shift in (4 - rows, -16, 0, 16, rows - 4):
        assert call(**{first: call.at[second] + shift}) == -1, shift


def test_in_place_counts_that_are_one(call):
    assert call(in_place=True, dropped=call.at["kept"]) == -1


def test_disjoint_ones_get_past_the_checks(call):
    """The launch itself fails without a GPU (PKV_ECUDA), or is refused by no check."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("host pointers are for a machine without a GPU")
    assert call() == -3 and call(in_place=True) == -3
    assert call(new=call.at["kept_out"] + 4 * BATCH) == -3 and call(dropped_out=call.at["kept_out"] - 4 * BATCH) == -3
    assert call(in_place=True, kept=call.at["dropped"] + 4 * BATCH) == -3
