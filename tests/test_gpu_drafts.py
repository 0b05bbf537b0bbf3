"""Drafted tokens and the latent cache on the GPU against the float64 oracle: masks, lengths, heads and blocks where
they can go wrong, errors that only the GPU sees, and a run of the calls as a decoder makes them."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_175_gb300 as pkv
from gpu_common import BAR_F32_RELL2, DEV, check_attention, err_flag, f64, rel_l2
from oracle import drafts as od

pytestmark = pytest.mark.gpu


def bf16(rng, *shape):
    return torch.as_tensor(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def trees(rng, ns, words):
    """Masks of random trees (ancestors and the token itself), as int64 words."""
    out = []
    for n in ns:
        m = []
        for i in range(n):
            p = int(rng.integers(-1, i)) if rng.random() < 0.6 else i - 1
            m.append((m[p] if p >= 0 else 0) | 1 << i)
        out += [[(x >> 64 * w) & (1 << 64) - 1 for w in range(words)] for x in m]
    return np.array(out, dtype=np.uint64).astype(np.int64).reshape(-1, words)


class Case:
    """Inputs of one attention call; kind (n_kv, d) for K / V pools, or (latent, rope) for a latent cache."""

    def __init__(self, kind, n_h, bs, ctx, ns, seed, mask="tree", extra=5):
        rng = np.random.default_rng(seed)
        self.latent = kind[1] in (32,) or kind[0] in (256, 512)
        self.kind, self.n_h, self.bs = kind, n_h, bs
        self.ctx, self.ns = np.asarray(ctx, np.int32), np.asarray(ns, np.int64)
        self.start = np.concatenate([[0], np.cumsum(self.ns)]).astype(np.int32)
        T = int(self.start[-1])
        nb = -(-self.ctx // bs)
        self.blocks = int(nb.sum()) + extra
        perm = rng.permutation(self.blocks).astype(np.int32)
        self.bt = np.full((len(ctx), max(1, int(nb.max()))), -1, np.int32)
        at = 0
        for s, n in enumerate(nb):
            self.bt[s, :n] = perm[at:at + n]
            at += n
        words = max(1, -(-int(max(ns)) // 64))
        self.mask = trees(rng, ns, words) if mask == "tree" else mask
        if self.latent:
            self.w, self.v = kind[0] + kind[1], kind[0]
            self.pools = [bf16(rng, self.blocks, 1, bs, self.w)]
        else:
            self.w = self.v = kind[1]
            self.pools = [bf16(rng, self.blocks, kind[0], bs, kind[1]) for _ in "kv"]
        self.q = bf16(rng, T, n_h, self.w)
        self.scale = 1 / math.sqrt(self.w)

    def oracle(self, clean=False):
        pools = [np.nan_to_num(f64(p), posinf=0.0, neginf=0.0) if clean else f64(p) for p in self.pools]
        k = lambda s: od.paged(pools[0], self.bt[s], self.ctx[s], self.bs)  # noqa: E731
        v = (lambda s: k(s)[:, :, :self.v]) if self.latent else lambda s: od.paged(pools[1], self.bt[s], self.ctx[s], self.bs)
        return od.step_attention(f64(self.q), k, v, self.start, self.ctx, self.scale, self.mask)

    def run(self, dtype=torch.float32, expect=0, start="given", bt=None, ctx=None, **kw):
        err = err_flag()
        dev = lambda x: None if x is None else torch.as_tensor(x, device=DEV)  # noqa: E731
        args = dict(q_start=dev(self.start) if start == "given" else start, tree_mask=dev(self.mask), out_dtype=dtype, err=err, **kw)
        bt, ctx = dev(self.bt if bt is None else bt), dev(self.ctx if ctx is None else ctx)
        pools = [p.to(DEV) for p in self.pools]
        if self.latent:
            out = pkv.paged_latent_attn(self.q.to(DEV), pools[0][:, 0], self.kind[0], bt, ctx, self.scale, **args)
        else:
            out = pkv.paged_tree_attn(self.q.to(DEV), *pools, bt, ctx, self.scale, **args)
        torch.cuda.synchronize()
        assert int(err.item()) == expect, int(err.item())
        return out

    def single(self):
        """Whether a bf16 output of this case takes the softmax weights rounded to bf16 once: over 32 query rows per kv
        head and sequence on average (pkv.h)."""
        group = self.n_h if self.latent else self.n_h // self.kind[0]
        return self.q.shape[0] * group > 32 * len(self.ctx)

    def check(self, out, ref, what):
        ref, size = ref
        if out.dtype == torch.bfloat16 and self.single():
            # each weight is off by at most half a step of bf16, 2^-8 of it, and so is the sum that divides them:
            # 2^-7 sum p |v|; and the output's own rounding.  Fp32 sums of up to 2^14 rows of random signs: 2^-17
            # As both roundings are spread evenly over their step (2^-8 / sqrt 3 in the mean square): sqrt 2 of that
            got = f64(out)
            assert np.isfinite(got).all(), what
            assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -17) * size).all(), what
            assert rel_l2(got, ref) <= math.sqrt(2) * 2.0 ** -8 / math.sqrt(3), (what, rel_l2(got, ref))
        else:
            check_attention(out, ref, what)


KV = [((2, 128), 8), ((1, 64), 7), ((3, 64), 24), ((1, 128), 64), ((8, 128), 8)]
LATENT = [((512, 64), 16), ((512, 64), 5), ((256, 64), 40), ((512, 32), 128), ((256, 32), 1)]
KINDS = [pytest.param(k, h, id=f"{k[0]}_{k[1]}_h{h}") for k, h in KV + LATENT]
BOTH = [pytest.param(k, h, id=f"{k[0]}_{k[1]}_h{h}") for k, h in (KV[0], LATENT[0])]


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("kind,n_h", KINDS)
def test_ragged_trees(kind, n_h, bs):
    # contexts and trees that end inside blocks, on their edges and on those of 64 and 128 rows; trees of no, one and
    # many tokens; nothing but the tree cached; a sequence of length 0
    ctx = [0, 1, bs, 5, 64, 65, 128 + 9, 300, 17, 129, 1030]
    ns = [0, 1, 2, 5, 1, 9, 10, 0, 17, 3, 7]
    c = Case(kind, n_h, bs, ctx, ns, seed=bs + n_h)
    ref = c.oracle()
    for dtype in (torch.float32, torch.bfloat16):
        c.check(c.run(dtype), ref, f"{kind} {n_h} {bs} {dtype}")


@pytest.mark.parametrize("kind,n_h", BOTH)
@pytest.mark.parametrize("n", [1, 3, 64, 70, 150])
def test_chains_and_wide_trees(kind, n_h, n):
    ctx = [n, n + 1, 2 * n + 63, 500]
    for mask in (None, "tree"):
        c = Case(kind, n_h, 16, ctx, [n] * 4, seed=n, mask=mask)
        out = c.run(start=None)
        c.check(out, c.oracle(), f"{kind} n{n} {mask}")
        assert torch.equal(out, c.run())                        # q_start that says the same
        c.check(c.run(torch.bfloat16), c.oracle(), f"{kind} n{n} {mask} bf16")


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_masks_that_leave_rows_empty_and_masks_short_of_words(kind, n_h):
    c = Case(kind, n_h, 16, [4, 90, 6], [4, 70, 3], seed=3)
    c.mask = c.mask[:, :1].copy()                                # tokens past 64 are attended by none
    c.mask[:4] = 0                                              # nothing but the tree cached: nothing attended
    c.mask[[5, 40]] = 0                                         # only the rows before the tree
    c.mask[6] = -1
    out = c.run()
    c.check(out, c.oracle(), "masks")
    assert not f64(out)[:4].any()


@pytest.mark.parametrize("kind,n_h", KINDS)
def test_values_that_nobody_attends_to_do_not_leak(kind, n_h):
    c = Case(kind, n_h, 32, [37, 130, 250, 1, 64], [5, 4, 10, 1, 0], seed=9)
    c.mask[5:9] &= ~np.int64(4)                                 # token 2 of sequence 1: padding, its row never written
    nasty = [float("nan"), float("inf"), -float("inf")]
    for s, n in enumerate(c.ctx):
        for p in c.pools:
            if n % 32:
                p[c.bt[s, n // 32], :, n % 32:] = nasty[s % 3]
    t = 130 - 4 + 2
    for p in c.pools:
        p[c.bt[1, t // 32], :, t % 32] = nasty[1]
    used = c.bt[c.bt >= 0]
    for p in c.pools:
        p[np.setdiff1d(np.arange(c.blocks), used)] = nasty[0]
    c.check(c.run(), c.oracle(clean=True), "stale rows")
    c.check(c.run(torch.bfloat16), c.oracle(clean=True), "stale rows bf16")


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_keys_of_masked_tokens_may_hold_anything(kind, n_h):
    # a masked key that is no number, with finite values: only where the values are the key itself can it not be
    if kind[0] == 512:
        pytest.skip("a latent row is key and value")
    c = Case(kind, n_h, 16, [50], [4], seed=4)
    c.mask[:, 0] = [1, 3, 5, 9]                                 # a root and three leaves
    c.pools[0][c.bt[0, 49 // 16], :, 49 % 16] = float("nan")    # the last leaf's key
    out, ref = f64(c.run()), c.oracle(clean=True)[0]
    assert np.abs(out[:3] - ref[:3]).max() <= 5e-4 and np.isnan(out[3]).all()


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_tokens_of_no_sequence_are_left_as_they_were(kind, n_h):
    c = Case(kind, n_h, 16, [40, 30], [3, 2], seed=5)
    c.q = torch.cat([c.q[:2], c.q, c.q[:3]])
    c.mask = np.concatenate([c.mask[:2], c.mask, c.mask[:3]])
    c.start = c.start + 2
    ref, size = c.oracle()
    out = torch.full((10, n_h, c.v), 7.0, device=DEV)
    c.run(out=out)
    got = f64(out)
    assert (got[:2] == 7).all() and (got[7:] == 7).all() and np.isnan(ref[7:]).all()
    assert rel_l2(got[2:7], ref[2:7]) <= BAR_F32_RELL2


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_errors_that_only_the_gpu_sees(kind, n_h):
    c = Case(kind, n_h, 16, [40, 30, 50], [3, 2, 4], seed=6)
    good = c.run()
    # a block id out of range: its rows contribute nothing
    bad = c.bt.copy()
    bad[1, 0] = c.blocks + 3
    out = c.run(bt=bad, expect=pkv.DEV_BAD_BLOCK)
    assert torch.equal(out[:3], good[:3]) and torch.equal(out[5:], good[5:])
    d = Case(kind, n_h, 16, [40, 30, 50], [3, 2, 4], seed=6)
    pools = [f64(p) for p in d.pools]
    k = lambda s: od.paged(pools[0], c.bt[s], c.ctx[s], 16)[:, 16 if s == 1 else 0:]  # noqa: E731
    v = (lambda s: k(s)[:, :, :c.v]) if c.latent else lambda s: od.paged(pools[1], c.bt[s], c.ctx[s], 16)[:, 16 if s == 1 else 0:]
    ref, _ = od.step_attention(f64(c.q), k, v, c.start, [40, 14, 50], c.scale, c.mask)
    assert rel_l2(f64(out), ref) <= BAR_F32_RELL2
    # a length past the table is cut to it, a negative one is none
    out = c.run(ctx=np.array([40, -5, 50], np.int32), expect=pkv.DEV_BAD_CTX)
    assert not f64(out[3:5]).any() and torch.equal(out[:3], good[:3])
    # starts out of order or range: no tokens there
    for start in ([0, 5, 3, 9], [0, 3, 12, 9], [-2, 3, 5, 9]):
        before = torch.full_like(good, 3.0)
        out = c.run(start=torch.tensor(start, dtype=torch.int32, device=DEV), out=before, expect=pkv.DEV_BAD_TREE)
        assert np.isfinite(f64(out)).all()
    # more tokens than rows: the first ones' rows are missing
    ctx = np.array([40, 1, 50], np.int32)
    out = c.run(ctx=ctx, expect=pkv.DEV_BAD_TREE)
    assert torch.equal(out[:3], good[:3])
    c.ctx = ctx
    ref, _ = c.oracle()
    assert rel_l2(f64(out), ref) <= BAR_F32_RELL2


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_many_sequences_and_long_ones(kind, n_h):
    rng = np.random.default_rng(1)
    ns = rng.integers(0, 4, size=700)
    c = Case(kind, n_h, 16, ns + rng.integers(0, 60, size=700) * (rng.random(700) < 0.8), ns, seed=7)
    c.check(c.run(), c.oracle(), "700 sequences")
    for ctx, ns in (([20011], [3]), ([9000, 3, 12345], [5, 3, 1])):
        c = Case(kind, n_h, 32, ctx, ns, seed=8)
        c.check(c.run(), c.oracle(), str(ctx))
        c.check(c.run(torch.bfloat16), c.oracle(), str(ctx))


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_results_depend_on_the_rows_alone(kind, n_h):
    c = Case(kind, n_h, 16, [700, 33, 1500], [6, 4, 9], seed=11)
    a = c.run()
    assert torch.equal(a, c.run())
    perm = np.random.default_rng(2).permutation(c.blocks)
    c.pools = [p[perm] for p in c.pools]
    c.bt = np.where(c.bt >= 0, np.argsort(perm)[np.maximum(c.bt, 0)], -1).astype(np.int32)
    assert torch.equal(a, c.run())


def test_one_token_is_decode_attention():
    c = Case((2, 128), 8, 16, [1, 100, 777], [1, 1, 1], seed=12, mask=None)
    a = c.run()
    b = pkv.paged_decode_attn(c.q.to(DEV), *(p.to(DEV) for p in c.pools), torch.as_tensor(c.bt, device=DEV), torch.as_tensor(c.ctx, device=DEV),
                              c.scale, out_dtype=torch.float32)
    assert rel_l2(f64(a), f64(b)) <= BAR_F32_RELL2


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_large_scores_and_offsets(kind, n_h):
    # scores that rise by far more than the lazy offset allows, along the context, in some heads only
    c = Case(kind, n_h, 16, [600, 64], [5, 2], seed=13)
    k = c.pools[0].float()
    for t in range(0, 600, 50):
        k[c.bt[0, t // 16], :, t % 16] *= 1 + t / 40
    c.pools[0] = k.to(torch.bfloat16)
    c.q[:, ::2] *= 4
    ref, size = c.oracle()
    got = f64(c.run())
    # a score is an fp32 sum of w products, off by at most w 2^-23 (a step per sum, also where it is cut off) of the sum of their
    # sizes; a weight by that, and so is their sum: twice it, and p's two parts 2^-16
    worst = max(float((np.abs(f64(c.q)[c.start[s]:c.start[s + 1]]).reshape(-1, c.w)
                       @ np.abs(od.paged(f64(c.pools[0]), c.bt[s], c.ctx[s], 16)).reshape(-1, c.w).T).max()) for s in range(2))
    off = c.w * 2.0 ** -23 * c.scale * worst
    assert off < 0.1 and np.isfinite(got).all() and (np.abs(got - ref) <= (2 * off + 2.0 ** -16) * size + 1e-6).all()


# ---- latent_append ------------------------------------------------------------------------------------
@pytest.mark.parametrize("latent,rope,n_h,inter", [(512, 64, 16, False), (512, 64, 128, True), (256, 64, 3, False), (512, 32, 33, True), (256, 32, 1, False)])
@pytest.mark.parametrize("n", [1, 7, 300])
def test_latent_append(latent, rope, n_h, inter, n):
    rng = np.random.default_rng(n + rope)
    w, bs, blocks = latent + rope, 32, 12
    wide, q = bf16(rng, n, w + 24), bf16(rng, n, n_h, 40 + rope)
    kv, cache, weight = wide[:, 8:8 + w], bf16(rng, blocks, bs, w), bf16(rng, latent)
    pos = rng.integers(-10 ** 6, 10 ** 6, size=n).astype(np.int32)
    slots = rng.choice(blocks * bs, size=n, replace=False).astype(np.int64)
    if n > 2:
        slots[1] = -1                                           # padding
    freqs, amp = oracle.rope_frequencies(rope, base=50000.0, scaling="yarn", factor=4.0, original_len=4096.0)
    table = pkv.rope_table(64, rope, base=50000.0, interleaved=inter, scaling="yarn", factor=4.0, original_len=4096.0)
    for wt in (weight, None):
        err, q_abs, dc = err_flag(), torch.full((n, n_h, w), 5.0, dtype=torch.bfloat16, device=DEV), cache.to(DEV)
        dq = q.to(DEV)
        pkv.latent_append(wide.to(DEV)[:, 8:8 + w], dq[..., 40:], torch.as_tensor(pos, device=DEV), torch.as_tensor(slots, device=DEV), table, dc,
                          q_out=q_abs[..., latent:], weight=None if wt is None else wt.to(DEV), eps=1e-5, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        here = slots >= 0
        ref_q = oracle.rope_tokens(f64(q)[..., 40:], pos, freqs, amp, interleaved=inter)
        ref_c = od.latent_rows(f64(kv), latent, pos, freqs, amp, inter, None if wt is None else f64(wt), 1e-5)
        want = f64(cache).reshape(-1, w).copy()
        got = f64(dc).reshape(-1, w)
        untouched = np.setdiff1d(np.arange(blocks * bs), slots)
        assert np.array_equal(got[untouched], want[untouched])
        # bf16's half step of the value; the fp32 arithmetic: a root, a quotient and two products of 2^-24 each after a sum
        # of 512 squares (9 levels of a tree and 16 in a row: 2^-19.3): 2^-18; of the rotation as for the rotary append, 2^-20 of the pair
        g, r = got[slots[here]], ref_c[here]
        assert (np.abs(g[:, :latent] - r[:, :latent]) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(r[:, :latent])).all()
        for x, y, src in ((g[:, latent:], r[:, latent:], f64(kv)[here, latent:]), (f64(q_abs)[here][..., latent:], ref_q[here], f64(q)[here][..., 40:])):
            mag = amp * math.sqrt(2) * np.abs(src).max(axis=-1, keepdims=True)
            assert (np.abs(x - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * mag).all()
        assert (f64(q_abs)[..., :latent] == 5).all() and (f64(q_abs)[~here] == 5).all()
        # in place, with a tensor of its own size: the same rows
        own = dq[..., 40:].contiguous()
        pkv.latent_append(wide.to(DEV)[:, 8:8 + w], own, torch.as_tensor(pos, device=DEV), torch.as_tensor(slots, device=DEV), table, cache.to(DEV), q_out=own)
        assert torch.equal(own[here], q_abs[here][..., latent:])


def test_latent_append_bad_slot():
    err, cache = err_flag(), torch.zeros(2, 16, 576, dtype=torch.bfloat16, device=DEV)
    kv, q = torch.ones(3, 576, dtype=torch.bfloat16, device=DEV), torch.ones(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    pkv.latent_append(kv, q, torch.zeros(3, dtype=torch.int32, device=DEV), torch.tensor([4, 32, 31], device=DEV), pkv.rope_table(64), cache, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pkv.DEV_BAD_SLOT
    rows = cache.view(-1, 576)
    assert (rows[[4, 31]] == 1).all() and rows.abs().sum() == 2 * 576


# ---- kv_tree_accept -----------------------------------------------------------------------------------
@pytest.mark.parametrize("shape", [(2, 128), (1, 64), (5, 64), (None, 576), (None, 288)])
@pytest.mark.parametrize("pools,bs", [(1, 64), (6, 16), (300, 32)])
def test_accept(shape, pools, bs):
    rng = np.random.default_rng(pools + bs)
    heads, w = shape
    if pools == 300 and w * (heads or 1) > 320:
        pytest.skip("small rows are enough for many caches")
    ns = np.array([0, 1, 5, 30, 64, 7, 9, 12])
    ctx = np.array([0, 1, 5, 97, 64 + 16, 40, 30, 300]) + np.array([0, 0, 0, 0, 33, 0, 0, 0])
    nb = -(-ctx // bs)
    blocks = int(nb.sum()) + 2
    perm, bt, at = rng.permutation(blocks), np.full((8, int(nb.max())), -1, np.int32), 0
    for s in range(8):
        bt[s, :nb[s]] = perm[at:at + nb[s]]
        at += nb[s]
    path, count = np.full((8, 70), 99, np.int32), np.zeros(8, np.int32)
    want = [[], [0], [0, 1, 2, 3, 4], np.sort(rng.permutation(30)[:17]), np.arange(1, 64, 2), [], [8], [2, 3, 9]]
    for s, p in enumerate(want):
        path[s, :len(p)], count[s] = p, len(p)
    caches = [bf16(rng, *((blocks, bs, w) if heads is None else (blocks, heads, bs, w))) for _ in range(min(pools, 6))]
    dev = [caches[i % len(caches)].to(DEV) for i in range(pools)]
    dev = [d.clone() for d in dev]
    err = err_flag()
    start = torch.as_tensor(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32), device=DEV)
    to = lambda x: torch.as_tensor(x.astype(np.int32), device=DEV)  # noqa: E731
    lens = pkv.kv_tree_accept(dev, to(bt), to(ctx), start, to(path), to(count), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert lens.tolist() == [int(c - n + len(p)) for c, n, p in zip(ctx, ns, want)]
    for i in sorted({0, len(caches) - 1, pools - 1}):
        ref = f64(caches[i % len(caches)])
        ref = ref[:, None] if heads is None else ref
        for s in range(8):
            ref, _ = od.accept(ref, bt[s], ctx[s], ns[s], list(want[s]), bs)
        assert np.array_equal(f64(dev[i]).reshape(ref.shape), ref), i


def test_accept_errors():
    rng = np.random.default_rng(0)
    bt = np.arange(12, dtype=np.int32).reshape(3, 4)
    pool = bf16(rng, 12, 2, 16, 64)
    ctx, to = np.array([50, 60, 5], np.int32), lambda x: torch.as_tensor(np.asarray(x, np.int32), device=DEV)  # noqa: E731

    def go(path, count, bt=bt, ctx=ctx, n=6, **kw):
        err, p = err_flag(), pool.to(DEV)
        lens = pkv.kv_tree_accept([p], to(bt), to(ctx), None, to(path), to(count), n_tok=3 * n, err=err, **kw)
        torch.cuda.synchronize()
        return lens.tolist(), int(err.item()), f64(p)

    T = pkv.DEV_BAD_TREE
    ok = [[1, 3], [0, 2], [0, 0]]
    lens, err, p = go(ok, [2, 2, 0])
    assert lens == [46, 56, 5] and err == T                      # six drafted tokens, five rows: as it was
    ctx = np.array([50, 60, 6], np.int32)
    assert go(ok, [2, 2, 0], ctx=ctx)[:2] == ([46, 56, 0], 0)
    for path, count, want in (([[3, 3], [0, 2], [0, 0]], [2, 2, 0], [45, 56, 0]),       # not ascending
                              ([[1, 6], [0, 2], [0, 0]], [2, 2, 0], [45, 56, 0]),       # past the tokens
                              ([[-1, 6], [0, 2], [0, 0]], [2, 2, 0], [44, 56, 0]),
                              ([[1, 3], [0, 2], [0, 0]], [3, -1, 0], [46, 54, 0])):     # counts out of range
        lens, err, p = go(path, count, ctx=ctx)
        assert lens == want and err == T, (path, lens, err)
    bad = bt.copy()
    bad[0, 2] = 12
    lens, err, p = go(ok, [2, 2, 0], bt=bad, ctx=ctx)
    assert lens == [46, 56, 0] and err == pkv.DEV_BAD_BLOCK
    ref, _ = od.accept(f64(pool), bt[1], 60, 6, [0, 2], 16)      # sequence 0's rows 44.. lie in that block
    assert np.array_equal(p, ref)
    lens = to(ctx)
    with pytest.raises(pkv.PkvError):
        pkv.kv_tree_accept([pool.to(DEV)], to(bt), lens, None, to(ok), to([2, 2, 0]), n_tok=18, new_lens=lens)


# ---- the calls together -------------------------------------------------------------------------------
def test_a_tree_step_is_the_decode_steps_of_its_path():
    """Append a tree, attend, accept a path, go on: the path's outputs and the cache are those of decode steps."""
    rng = np.random.default_rng(21)
    n_h, n_kv, d, bs, B, n, have = 8, 2, 128, 16, 3, 7, [20, 33, 47]
    parents = [-1, 0, 0, 1, 2, 4, 3]
    depth = [0, 1, 1, 2, 2, 3, 3]
    path = [0, 2, 4, 5]
    anc = []
    for i, p in enumerate(parents):
        anc.append((anc[p] if p >= 0 else 0) | 1 << i)
    table, bt = pkv.rope_table(d), np.arange(B * 5, dtype=np.int32).reshape(B, 5)
    kp, vp = (bf16(rng, B * 5, n_kv, bs, d).to(DEV) for _ in "kv")
    qkv = bf16(rng, B * n, (n_h + 2 * n_kv) * d).to(DEV)
    q, k, v = (x.view(B * n, -1, d) for x in qkv.split([n_h * d, n_kv * d, n_kv * d], 1))
    to = lambda x, t=torch.int32: torch.as_tensor(np.asarray(x), device=DEV).to(t)  # noqa: E731
    rows = np.array([[h + i for i in range(n)] for h in have])
    slots = to(bt[np.arange(B)[:, None], rows // bs].astype(np.int64) * bs + rows % bs, torch.int64).flatten()
    pos = to([[h + z for z in depth] for h in have]).flatten()
    k1, v1, k2, v2 = kp.clone(), vp.clone(), kp.clone(), vp.clone()
    q1 = pkv.rope_append(q, k, v, pos, slots, table, k1, v1)
    out = pkv.paged_tree_attn(q1, k1, v1, to(bt), to(have) + n, d ** -0.5, tree_mask=to([[a] for a in anc] * B, torch.int64), out_dtype=torch.float32)
    lens = pkv.kv_tree_accept([k1, v1], to(bt), to(have) + n, None, to([path] * B), to([len(path)] * B), n_tok=B * n)
    assert lens.tolist() == [h + 4 for h in have]
    for i, node in enumerate(path):                              # the same tokens one step at a time
        at = torch.arange(B, device=DEV) * n + node
        r = np.array(have) + i
        step = to(bt[np.arange(B), r // bs].astype(np.int64) * bs + r % bs, torch.int64)
        qs = pkv.rope_append(q[at].contiguous(), k[at].contiguous(), v[at].contiguous(), to(r), step, table, k2, v2)
        o = pkv.paged_decode_attn(qs, k2, v2, to(bt), to(r + 1), d ** -0.5, out_dtype=torch.float32)
        assert rel_l2(f64(out[at]), f64(o)) <= BAR_F32_RELL2, node
    for b, h in enumerate(have):
        for a, z in ((k1, k2), (v1, v2)):
            row = lambda p: p[bt[b]].transpose(0, 1).flatten(1, 2)[:, :h + 4]  # noqa: E731,B023
            assert torch.equal(row(a), row(z))


def test_latent_tree_step():
    """The same over a latent cache: append, attend, accept, and one more token."""
    rng = np.random.default_rng(22)
    n_h, latent, rope, bs, B, n, have = 16, 512, 64, 32, 2, 5, [40, 63]
    w, table, bt = latent + rope, pkv.rope_table(64), np.arange(8, dtype=np.int32).reshape(2, 4)
    caches = [bf16(rng, 8, bs, w).to(DEV) for _ in range(2)]
    to = lambda x, t=torch.int32: torch.as_tensor(np.asarray(x), device=DEV).to(t)  # noqa: E731
    anc, depth, path = [1, 3, 5, 11, 21], [0, 1, 1, 2, 2], [0, 2, 4]
    weight = bf16(rng, latent).to(DEV)

    def step(cache, toks, rows, pos, mask):
        m = len(toks)
        slots = to(bt[np.arange(B)[:, None], rows // bs].astype(np.int64) * bs + rows % bs, torch.int64).flatten()
        at = (torch.arange(B, device=DEV)[:, None] * n + to(toks, torch.int64)).flatten()
        q = q_abs[at].clone()
        pkv.latent_append(kv[at], q_pe[at], to(pos).flatten(), slots, table, cache, q_out=q[..., latent:], weight=weight)
        return pkv.paged_latent_attn(q, cache, latent, to(bt), to(rows[:, 0]) + m, w ** -0.5, tree_mask=mask, out_dtype=torch.float32)

    kv, q_abs, q_pe = bf16(rng, B * n, w).to(DEV), bf16(rng, B * n, n_h, w).to(DEV), bf16(rng, B * n, n_h, rope).to(DEV)
    h = np.array(have)[:, None]
    one, two = caches[0].clone(), caches[0].clone()
    out = step(one, range(n), h + np.arange(n), h + np.array(depth), to([[a] for a in anc] * B, torch.int64))
    lens = pkv.kv_tree_accept([one], to(bt), to(have) + n, None, to([path] * B), to([3] * B), n_tok=B * n)
    assert lens.tolist() == [x + 3 for x in have]
    for i, node in enumerate(path):
        o = step(two, [node], h + i, h + i, None)
        assert rel_l2(f64(out.view(B, n, n_h, latent)[:, node]), f64(o)) <= BAR_F32_RELL2, node
    for b, x in enumerate(have):
        assert torch.equal(one[bt[b]].flatten(0, 1)[:x + 3], two[bt[b]].flatten(0, 1)[:x + 3])


@pytest.mark.parametrize("kind,n_h", BOTH)
def test_captured_calls_follow_their_inputs(kind, n_h):
    c = Case(kind, n_h, 16, [300, 90], [4, 4], seed=31, mask=None)
    pools = [p.to(DEV) for p in c.pools]
    bt, ctx, q, out = torch.as_tensor(c.bt, device=DEV), torch.as_tensor(c.ctx, device=DEV), c.q.to(DEV), torch.empty(8, n_h, c.v, device=DEV)
    start = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    path, count, lens = torch.tensor([[0, 2, 3]] * 2, dtype=torch.int32, device=DEV), torch.tensor([3, 2], dtype=torch.int32, device=DEV), ctx.clone()

    def step():
        if c.latent:
            pkv.paged_latent_attn(q, pools[0][:, 0], kind[0], bt, ctx, c.scale, q_start=start, out=out)
        else:
            pkv.paged_tree_attn(q, *pools, bt, ctx, c.scale, q_start=start, out=out)
        pkv.kv_tree_accept(pools, bt, ctx, start, path, count, new_lens=lens)

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        step()
    for p, x in zip(pools, c.pools):
        p.copy_(x)
    for a, b, lo in (([300, 90], [0, 4, 8], 0), ([100, 50], [0, 1, 8], 0), ([17, 9], [2, 5, 8], 2)):
        ctx.copy_(torch.tensor(a, dtype=torch.int32))
        start.copy_(torch.tensor(b, dtype=torch.int32))
        for p, x in zip(pools, c.pools):
            p.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        c.ctx, c.start = np.array(a, np.int32), np.array(b, np.int32)
        ref, _ = c.oracle()
        assert rel_l2(f64(out)[lo:], ref[lo:]) <= BAR_F32_RELL2
        for i, n in enumerate(np.diff(b)):                       # a path ends at the first entry that is no token
            kept = [p for p in [0, 2, 3][:min(int(count[i]), n)] if p < n]
            assert int(lens[i]) == a[i] - n + len(kept)
