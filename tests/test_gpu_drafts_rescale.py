"""Offsets that are raised within a piece, several times: sums and accumulators are rescaled in place, for query rows whose own
maximum has hardly moved, too.  Blocks with a bad id at the start of a tile, and trees over several tiles."""
import numpy as np
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv
from drafts_common import check, reference
from test_gpu_drafts import Case

pytestmark = pytest.mark.gpu
DTYPES = (torch.float32, torch.bfloat16)
# kind, heads, tokens per sequence, sequences: lines of some 2000 tiles, a dozen or more for each CTA, and row tiles of 16, 32
# and 64 query rows (bf16) or of 16 and 32 (fp32)
STEPS = [pytest.param(*x, id=f"{x[0][0]}_{x[0][1]}_h{x[1]}_n{x[2]}") for x in
         [((8, 128), 32, 2, 12), ((8, 128), 32, 6, 12), ((8, 128), 32, 12, 12), ((8, 64), 32, 2, 12), ((8, 64), 32, 6, 12), ((8, 64), 32, 12, 12),
          ((512, 64), 16, 1, 40), ((512, 64), 16, 2, 40), ((512, 64), 32, 3, 40), ((256, 64), 16, 1, 40), ((256, 32), 16, 2, 40), ((256, 64), 64, 2, 40)]]


def rising(kind, n_h, n, batch, seed, bs=16):
    """A third of the heads see scores that rise by 9 (base 2) every 64 rows, a third that fall, and a third neither: each tile of a softmax
    group of the K / V kernel and every fourth of the latent one raises the offsets of all query rows by more than 2^32."""
    rng = np.random.default_rng(seed)
    ctx = rng.integers(2000, 3500, size=batch)
    c = Case(kind, n_h, bs, ctx, [n] * batch, seed=seed, mask=None)
    step = 9 / (c.scale * 1.4426950408889634)
    c.q[..., -1] = 0.0
    c.q[:, ::3, -1], c.q[:, 1::3, -1] = step, -step
    for s, L in enumerate(ctx):
        t = np.arange(L)
        c.pools[0][c.bt[s, t // bs], :, t % bs, -1] = torch.as_tensor(t // 64).to(torch.bfloat16)[:, None]
    return c


@pytest.mark.parametrize("kind,n_h,n,batch", STEPS)
def test_scores_that_rise_along_the_context(kind, n_h, n, batch):
    c = rising(kind, n_h, n, batch, seed=n_h + n)
    ref = reference(c)
    for dtype in DTYPES:
        check(c.run(dtype), ref, "rising")


@pytest.mark.parametrize("kind,n_h,n,batch", [STEPS[1], STEPS[5], STEPS[7], STEPS[8]])
def test_bad_blocks_at_the_start_of_tiles(kind, n_h, n, batch):
    c = rising(kind, n_h, n, batch, seed=3)
    bt, per = c.bt.copy(), (64 if c.latent else 128) // 16
    rng = np.random.default_rng(4)
    for s in range(batch):
        tiles = -(-int(c.ctx[s]) // (16 * per))
        bt[s, 0] = c.blocks + 5
        bt[s, per * rng.integers(1, tiles - 1, size=3)] = -7
        if s % 3 == 0:
            bt[s, :2 * per] = c.blocks                         # whole tiles of them
    ref = reference(c, bt)
    for dtype in DTYPES:
        check(c.run(dtype, bt=bt, expect=pkv.DEV_BAD_BLOCK), ref, "bad blocks")


@pytest.mark.parametrize("mask", ["tree", None])
@pytest.mark.parametrize("kind,n_h", [pytest.param(k, h, id=f"{k[0]}_{k[1]}_h{h}") for k, h in [((2, 128), 2), ((1, 64), 3), ((256, 32), 2)]])
def test_trees_of_several_tiles(kind, n_h, mask):
    for n in (300, 700):
        c = Case(kind, n_h, 16, [n, n + 900, 2 * n + 77, n + 40] * 2, [n, n - 3, n, n - 150] * 2, seed=n, mask=mask)
        ref = reference(c)
        for dtype in DTYPES:
            check(c.run(dtype), ref, f"{n} {mask}")


@pytest.mark.parametrize("seed", range(12))
def test_random_steps_with_bad_blocks(seed):
    rng = np.random.default_rng(2000 + seed)
    if seed % 2:
        kind, n_h = (int(rng.choice([256, 512])), int(rng.choice([32, 64]))), int(rng.choice([1, 8, 16, 31, 64, 128]))
    else:
        n_kv = int(rng.choice([1, 2, 8]))
        kind, n_h = (n_kv, int(rng.choice([64, 128]))), n_kv * int(rng.choice([1, 2, 5, 16, 33]))
    batch, bs = int(rng.integers(1, 12)), int(rng.choice([16, 32, 64]))
    ns = rng.integers(1, int(rng.choice([2, 9, 33])) + 1, size=batch)
    ctx = np.array([int(n + 2.0 ** rng.uniform(0, 12)) for n in ns])
    c = Case(kind, n_h, bs, ctx, ns, seed=seed, mask="tree" if rng.random() < 0.7 else None)
    bt = c.bt.copy()
    hit = (rng.random(bt.shape) < 0.15) & (bt >= 0)
    hit[int(np.argmax(ctx)), 0] = True
    bt[hit] = rng.choice([-1, -9, c.blocks, 0x7fffffff], size=int(hit.sum()))
    ref = reference(c, bt)
    for dtype in DTYPES:
        check(c.run(dtype, bt=bt, expect=pkv.DEV_BAD_BLOCK), ref, f"{kind} {n_h} {ctx} {ns}")
