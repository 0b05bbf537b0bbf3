"""Attention of drafted tokens and over the latent cache at shapes where its partition, its row tiles or its address
arithmetic can go wrong, against the float64 oracle."""
import numpy as np
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv
from gpu_common import DEV, err_flag, f64
from test_gpu_drafts import BOTH, KV, LATENT, Case, bf16

pytestmark = pytest.mark.gpu
DTYPES = (torch.float32, torch.bfloat16)


def check_pairs(got, ref, size, what):
    """bf16 outputs of weights in two bf16 parts (2^-16 of each), fp32 sums (2^-17) and the output's own rounding, 2^-8 of
    it.  Outputs of one row are the row: at 4 half a step is 2^-6, so a bar of 10^-2 on the error itself does not fit them."""
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -16 + 2.0 ** -17) * size).all(), what


@pytest.mark.parametrize("kind,n_h", [pytest.param(k, h, id=f"{k[0]}_{k[1]}_h{h}") for k, h in
                                      [((1, 64), 64), ((1, 128), 50), ((2, 128), 34), ((512, 64), 128), ((512, 64), 33), ((256, 64), 70)]])
def test_teams_whose_members_lack_a_row_tile(kind, n_h):
    # rows of a sequence from less than one tile to many, so that a member of a team often has none; pieces that start in such
    # a segment
    rng = np.random.default_rng(n_h)
    ns = [1, 9, 2, 17, 1, 5, 1, 1, 3, 12]
    ctx = [int(n + rng.integers(0, 700)) for n in ns]
    c = Case(kind, n_h, 32, ctx, ns, seed=n_h)
    ref = c.oracle()
    for dtype in DTYPES:
        c.check(c.run(dtype), ref, f"{kind} {n_h} {dtype}")


@pytest.mark.parametrize("kind,n_h", BOTH)
@pytest.mark.parametrize("ctx", [[9000], [4100, 60], [64 * 152], [1] * 5 + [5000]])
def test_few_segments_of_many_parts(kind, n_h, ctx):
    for n in (1, 6):
        c = Case(kind, n_h, 64, ctx, [min(n, x) for x in ctx], seed=ctx[0] + n)
        ref = c.oracle()
        for dtype in DTYPES:
            c.check(c.run(dtype), ref, f"{kind} {ctx} {n} {dtype}")


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_one_table_for_short_and_long(kind, n_h):
    # the join is laid out by the table's width; lengths may be far below it
    c = Case(kind, n_h, 16, [30, 2, 300], [3, 2, 1], seed=4)
    wide = np.full((3, 5000), -1, np.int32)
    wide[:, :c.bt.shape[1]] = c.bt
    ref = c.oracle()
    for dtype in DTYPES:
        c.check(c.run(dtype, bt=wide), ref, f"{kind} {dtype}")


@pytest.mark.parametrize("kind,n_h", BOTH)
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(kind, n_h, scale):
    c = Case(kind, n_h, 16, [1, 200, 70, 128], [1, 9, 20, 0], seed=21)
    c.scale = scale if scale <= 0 else c.scale * scale
    c.check(c.run(), c.oracle(), f"{kind} scale {scale}")


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_scores_that_are_no_numbers_stay_in_their_rows(kind, n_h):
    # an infinite and a NaN query element: that token's head alone has no number
    c = Case(kind, n_h, 16, [300, 90], [4, 3], seed=22)
    clean = c.run()
    c.q[1, 2, 0], c.q[5, 0, 3] = float("nan"), float("nan")
    out = c.run()
    bad = torch.zeros(out.shape[:2], dtype=torch.bool)
    bad[1, 2] = bad[5, 0] = True
    assert torch.isnan(out[bad.to(DEV)]).all() and torch.equal(out[~bad.to(DEV)], clean[~bad.to(DEV)])


@pytest.mark.parametrize("latent", [False, True])
def test_blocks_behind_two_to_the_31_elements(latent):
    # the sequence's blocks are the pool's last ones, behind 2^32 bytes and 2^31 elements
    kind, n_h, bs = ((512, 64), 16, 64) if latent else ((8, 128), 32, 64)
    c = Case(kind, n_h, bs, [500, 77], [5, 2], seed=23)
    block = bs * (c.w if latent else kind[0] * kind[1])
    far = (1 << 31) // block + 3
    pools = [torch.empty(far + c.blocks, *p.shape[1:], dtype=torch.bfloat16, device=DEV) for p in c.pools]
    for big, p in zip(pools, c.pools):
        big[far:].copy_(p)
    bt = torch.as_tensor(np.where(c.bt >= 0, c.bt + far, -1).astype(np.int32), device=DEV)
    args = dict(q_start=torch.as_tensor(c.start, device=DEV), tree_mask=torch.as_tensor(c.mask, device=DEV), out_dtype=torch.float32)
    q, ctx, err = c.q.to(DEV), torch.as_tensor(c.ctx, device=DEV), err_flag()
    if latent:
        out = pkv.paged_latent_attn(q, pools[0][:, 0], 512, bt, ctx, c.scale, err=err, **args)
    else:
        out = pkv.paged_tree_attn(q, *pools, bt, ctx, c.scale, err=err, **args)
    c.check(out, c.oracle(), "far blocks")
    # the path 1, 3 of the first sequence's drafts, and the append of a token to the last slot
    path = torch.tensor([[1, 3], [0, 0]], dtype=torch.int32, device=DEV)
    shaped = [p[:, 0] for p in pools] if latent else pools
    lens = pkv.kv_tree_accept(shaped, bt, ctx, args["q_start"], path, torch.tensor([2, 1], dtype=torch.int32, device=DEV), err=err)
    assert lens.tolist() == [497, 76]
    row = lambda p, t: p[int(c.bt[0, t // bs]), :, t % bs]  # noqa: E731
    for big, p in zip(pools, c.pools):
        assert torch.equal(row(big[far:], 495).cpu(), row(p, 496)) and torch.equal(row(big[far:], 496).cpu(), row(p, 498))
    if latent:
        kv = bf16(np.random.default_rng(3), 1, c.w).to(DEV)
        slot = torch.tensor([(far + c.blocks) * bs - 1], device=DEV)
        pkv.latent_append(kv, q[:1, :, :64].contiguous(), torch.zeros(1, dtype=torch.int32, device=DEV), slot, pkv.rope_table(64), pools[0][:, 0], err=err)
        assert torch.equal(pools[0][-1, 0, -1], kv[0])          # position 0 turns nothing, no weight scales nothing
    assert int(err.item()) == 0


@pytest.mark.parametrize("kind,n_h", [pytest.param(*KV[1], id="kv"), pytest.param(*LATENT[2], id="latent")])
def test_nothing_to_do(kind, n_h):
    # no sequence has a cached row, or none has a token: zeros, or nothing at all
    c = Case(kind, n_h, 16, [0, 0, 0], [2, 0, 3], seed=24)
    for dtype in DTYPES:
        assert not c.run(dtype).any()
    c = Case(kind, n_h, 16, [50, 3], [0, 0], seed=25, mask=None)
    c.q = bf16(np.random.default_rng(1), 4, n_h, c.w)           # four tokens of no sequence
    out = torch.full((4, n_h, c.v), 7.0, device=DEV)
    c.run(out=out)
    assert bool((out == 7).all())


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_more_sequences_than_threads(kind, n_h):
    rng = np.random.default_rng(5)
    ctx = rng.integers(0, 40, size=1100)
    c = Case(kind, n_h, 16, ctx, np.minimum(ctx, 1), seed=26, mask=None)
    check_pairs(f64(c.run(torch.bfloat16)), *c.oracle(), "1100 sequences")




@pytest.mark.parametrize("seed", range(24))
def test_random_steps(seed):
    """Heads, blocks, lengths, trees and bad blocks at random."""
    rng = np.random.default_rng(1000 + seed)
    if seed % 2:
        kind, n_h = (int(rng.choice([256, 512])), int(rng.choice([32, 64]))), int(rng.choice([1, 3, 8, 16, 31, 64, 128]))
    else:
        n_kv = int(rng.choice([1, 2, 3, 8]))
        kind, n_h = (n_kv, int(rng.choice([64, 128]))), n_kv * int(rng.choice([1, 2, 5, 8, 16, 33, 64]))
    batch, most = int(rng.integers(1, 12)), int(rng.choice([1, 2, 9, 33]))
    ns = rng.integers(0, most + 1, size=batch)
    if ns.sum() == 0:
        ns[0] = 1
    ctx = [int(n + 2.0 ** rng.uniform(0, 11)) * int(rng.random() < 0.9) for n in ns]
    ctx = [max(c, int(n)) if c else 0 for c, n in zip(ctx, ns)]
    c = Case(kind, n_h, int(rng.choice([16, 32, 64])), ctx, ns, seed=seed, mask="tree" if rng.random() < 0.7 else None)
    ref = c.oracle()
    what = f"{kind} {n_h} {ctx} {ns}"
    c.check(c.run(), ref, what)
    if c.single():
        c.check(c.run(torch.bfloat16), ref, what)
    else:
        check_pairs(f64(c.run(torch.bfloat16)), *ref, what)


def test_a_long_append_is_its_parts():
    # more tokens than one dimension of the grid takes, against calls of a few thousand
    n, n_h, latent, rope, bs = 140003, 2, 256, 32, 64
    g = torch.Generator(device=DEV).manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    kv, q, weight, table = rnd(n, latent + rope), rnd(n, n_h, rope), rnd(latent), pkv.rope_table(64, rope)
    pos, blocks = torch.arange(n, dtype=torch.int32, device=DEV), -(-n // bs)
    slots, err = torch.randperm(blocks * bs, generator=g, device=DEV)[:n], err_flag()
    caches = [torch.zeros(blocks, bs, latent + rope, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    out = pkv.latent_append(kv, q, pos, slots, table, caches[0], weight=weight, err=err)
    parts = [pkv.latent_append(kv[i:i + 9001], q[i:i + 9001], pos[i:i + 9001], slots[i:i + 9001], table, caches[1], weight=weight, err=err)
             for i in range(0, n, 9001)]
    assert torch.equal(out, torch.cat(parts)) and torch.equal(*caches) and int(err.item()) == 0
    assert bool(caches[0].view(-1, latent + rope)[slots].any(1).all())
