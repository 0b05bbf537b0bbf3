"""Ranges of q_start that are out of order or range cost their own sequences' tokens and nobody else's."""
import numpy as np
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv
from drafts_common import check, reference
from gpu_common import DEV
from test_gpu_drafts import BOTH, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("start,good", [([0, 3, 12, 9], [(0, 0, 3)]), ([-2, 3, 5, 9], [(1, 3, 5), (2, 5, 9)]),
                                        ([0, 5, 3, 9], [(0, 0, 5), (2, 3, 9)]), ([4, 4, 2, 1], [(0, 4, 4)]),
                                        ([0, 3, 5, 0x7fffffff], [(0, 0, 3), (1, 3, 5)])])
@pytest.mark.parametrize("kind,n_h", BOTH)
def test_ranges_that_are_none(kind, n_h, start, good, dtype):
    c = Case(kind, n_h, 16, [40, 30, 50], [3, 2, 4], seed=6)
    out = torch.full((9, n_h, c.v), 3.0, dtype=dtype, device=DEV)
    c.run(dtype, start=torch.tensor(start, dtype=torch.int32, device=DEV), out=out, expect=pkv.DEV_BAD_TREE)
    full, touched = c.start, np.zeros(9, bool)
    for s, a, b in good:                                       # a sequence's own range, the others without tokens
        if a == b:
            continue
        c.start = np.array([a] * (s + 1) + [b] * (3 - s), np.int32)
        ref = [x.copy() for x in reference(c)]
        for s2, a2, b2 in good:
            if s2 > s:                                         # two ranges that share tokens: either's output may stay
                for x in ref:
                    x[max(a, a2):min(b, b2)] = np.nan
        for s2, a2, b2 in good:
            if s2 < s:
                for x in ref:
                    x[max(a, a2):min(b, b2)] = np.nan
        check(out, ref, f"{start} {s}")
        touched[a:b] = True
    c.start = full
    assert bool((out[torch.as_tensor(~touched, device=DEV)] == 3).all())
