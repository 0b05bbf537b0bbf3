"""The README's example of drafted tokens and of the latent cache, as it stands there."""
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv
from gpu_common import DEV, f64, rel_l2
from oracle import drafts as od

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_the_example():
    batch, n, n_h, n_kv, d, bs, latent, rope, blocks, lens = 3, 4, 8, 2, 64, 16, 256, 64, 24, [37, 16, 90]
    rng = np.random.default_rng(0)
    rnd = lambda *s: torch.as_tensor(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
    dev = lambda x, t=torch.int32: torch.as_tensor(np.asarray(x), device=DEV).to(t)  # noqa: E731
    bt = np.arange(batch * 8).reshape(batch, 8)
    depth = [0, 1, 1, 2]                                        # token 0, its children 1 and 2, and 3 under 2
    base = np.array(lens)
    place = lambda s, t: bt[s, t // bs] * bs + t % bs  # noqa: E731
    names = dict(
        torch=torch, pkv=pkv, latent=latent, rope=rope, scale=0.125, q=rnd(batch * n, n_h, d), k_new=rnd(batch * n, n_kv, d),
        v_new=rnd(batch * n, n_kv, d), depth_positions=dev([b + x for b in lens for x in depth]),
        draft_slots=dev([place(s, base[s] + i) for s in range(batch) for i in range(n)], torch.int64), table=pkv.rope_table(d),
        k_pool=rnd(blocks, n_kv, bs, d), v_pool=rnd(blocks, n_kv, bs, d), block_tables=dev(bt), context_lens=dev(base + n),
        q_start=dev(np.arange(batch + 1) * n), tree_mask=dev([[1], [3], [5], [13]] * batch, torch.int64),
        path=dev([[0, 2, 3]] * batch), n_accept=dev([3, 1, 2]), kv=rnd(batch, latent + rope), q_rope=rnd(batch, n_h, rope),
        positions=dev(base), slot_mapping=dev([place(s, base[s]) for s in range(batch)], torch.int64),
        latent_cache=rnd(blocks, bs, latent + rope), q_absorbed=rnd(batch, n_h, latent + rope), norm_weight=rnd(latent))
    code = next(b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "kv_tree_accept" in b)
    tree, rest = code.split("# ... the model picks")
    exec(tree, names)
    pools = [f64(names["k_pool"]), f64(names["v_pool"])]
    rows = lambda i: lambda s: od.paged(pools[i], bt[s], base[s] + n, bs)  # noqa: E731
    ref, _ = od.step_attention(f64(names["q_rot"]), rows(0), rows(1), np.arange(batch + 1) * n, base + n, 0.125,
                               f64(names["tree_mask"]).astype(np.int64))
    assert rel_l2(f64(names["out"]), ref) <= 2e-3
    exec("# ... " + rest, names)
    assert names["context_lens"].tolist() == [base[0] + 3, base[1] + 1, base[2] + 2]
    after = f64(names["k_pool"])
    row = lambda p, s, t: p[bt[s, t // bs], :, t % bs]  # noqa: E731
    assert np.array_equal(row(after, 0, base[0] + 1), row(pools[0], 0, base[0] + 2))
    assert np.array_equal(row(after, 0, base[0] + 2), row(pools[0], 0, base[0] + 3))
    assert np.array_equal(row(after, 1, base[1] + 1), row(pools[0], 1, base[1] + 1))
    cache, ctx = f64(names["latent_cache"])[:, None], names["context_lens"].tolist()
    k = lambda s: od.paged(cache, bt[s], ctx[s], bs)  # noqa: E731
    ref, _ = od.step_attention(f64(names["q_absorbed"]), k, lambda s: k(s)[:, :, :latent], np.arange(batch + 1), np.array(ctx), 0.125, None)
    assert rel_l2(f64(names["out"]), ref) <= 2e-3
    assert tuple(names["out"].shape) == (batch, n_h, latent)
