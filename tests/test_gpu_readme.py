"""The example of the README as it stands there, on sequences two of which share a prompt prefix."""
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def example():
    return next(b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "kv_evict" in b)


def test_the_example_cuts_what_is_alone_and_moves_no_shared_row():
    n_h, n_kv, d, bs, max_blocks, num_blocks, budget, recent = 8, 2, 64, 16, 8, 40, 32, 4
    g = torch.Generator().manual_seed(0)
    manager = pkv.BlockManager(num_blocks, bs)
    prefix = list(range(64))
    manager.add_sequence(0, prefix + [1] * 9)
    assert manager.add_sequence(1, prefix + [2] * 20)[1] == 64  # its first four blocks are sequence 0's
    manager.add_sequence(2, [3] * 70)
    manager.add_sequence(3, [4] * 20)                           # shorter than the budget
    sequences, batch = [0, 1, 2, 3], 4
    slots = manager.append_tokens(sequences, [9] * 4)
    tables, lens = manager.tables(sequences, max_blocks)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    names = dict(n_kv=n_kv, block_size=bs, head_dim=d, num_blocks=num_blocks, max_blocks=max_blocks, batch=batch, scale=d ** -0.5,
                 budget=budget, recent=recent, manager=manager, sequences=sequences, q=rnd(batch, n_h, d), k_new=rnd(batch, n_kv, d),
                 v_new=rnd(batch, n_kv, d), k_pool=rnd(num_blocks, n_kv, bs, d), v_pool=rnd(num_blocks, n_kv, bs, d),
                 slot_mapping=torch.as_tensor(slots, device=DEV), tail_seq=torch.arange(batch, dtype=torch.int32, device=DEV),
                 positions=torch.as_tensor(lens - 1, device=DEV), block_tables=torch.as_tensor(tables, device=DEV),
                 context_lens=torch.as_tensor(lens, device=DEV), keep=torch.full((batch,), budget, dtype=torch.int32, device=DEV))
    k_pool, v_pool = names["k_pool"], names["v_pool"]
    code = example()
    cut = code.index("state = ")
    exec(code[:cut], names)                                     # the appends
    torch.cuda.synchronize()
    before = [k_pool.clone(), v_pool.clone()]
    exec(code[cut:], names)
    torch.cuda.synchronize()
    assert names["context_lens"].tolist() == manager.tables(sequences, max_blocks)[1].tolist() == [74, 85, budget, 21]
    whole = np.unique(np.concatenate([tables[s, :-(-lens[s] // bs)] for s in (0, 1, 3)]))
    moved = tables[2, :budget // bs]
    for pool, was in zip((k_pool, v_pool), before):
        assert torch.equal(pool[whole], was[whole])             # nothing of the sequences that stay whole
        assert not torch.equal(pool[moved], was[moved])
    assert names["state"].kept.tolist() == [0, 0, budget, 0] and names["state"].dropped.tolist() == [0, 0, 71 - budget, 0]
