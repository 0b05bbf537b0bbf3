"""The rotary calls take a table from rope_table and nothing else of its size."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv

pytestmark = pytest.mark.gpu


class Other(ctypes.Structure):
    _fields_ = pkv.RopeTable._fields_


def not_tables():
    raw = bytes(pkv.rope_table(64))
    yield from (None, 0, raw, bytearray(raw), np.frombuffer(raw, np.uint8), Other.from_buffer_copy(raw), raw[:-8], pkv.RopeTable)


def test_only_a_table_is_read_as_one():
    q, k = (torch.randn(3, h, 64, device="cuda").to(torch.bfloat16) for h in (4, 2))
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    pos, slots, q_out = torch.arange(3, dtype=torch.int32, device="cuda"), torch.arange(3, device="cuda"), torch.full_like(q, 5.0)
    for bad in not_tables():
        with pytest.raises(pkv.PkvError, match="rope_table"):
            pkv.rope_qk(q, k, pos, bad, q_out=q_out)
        with pytest.raises(pkv.PkvError, match="rope_table"):
            pkv.rope_append(q, k, k, pos, slots, bad, pool, pool.clone(), q_out=q_out)
    torch.cuda.synchronize()
    assert bool((q_out == 5.0).all()) and not pool.any()
    assert not torch.equal(pkv.rope_qk(q, k, pos, pkv.rope_table(64))[0], q_out)
