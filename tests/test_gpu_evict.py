"""Accounted attention, eviction by the accounts, and the operators run together as a serving loop."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_175_gb300 as pkv
from gpu_common import DEV, check_attention, err_flag, f64
from oracle import evict as ev

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.as_tensor(x, device=DEV)


def pools(lens, n_kv, d, bs, seed, spare=3):
    rng = np.random.default_rng(seed)
    nb = [-(-int(n) // bs) for n in lens]
    blocks = sum(nb) + spare
    perm = rng.permutation(blocks).astype(np.int32)
    bt = np.full((len(lens), max(max(nb), 1)), -1, np.int32)
    cur = 0
    for s, n in enumerate(nb):
        bt[s, :n] = perm[cur:cur + n]
        cur += n
    g = torch.Generator().manual_seed(seed)
    kp, vp = (torch.randn(blocks, n_kv, bs, d, generator=g).to(torch.bfloat16) for _ in range(2))
    return kp, vp, bt, g


def run_mass(q, kp, vp, bt, lens, scale, mass, out_dtype=torch.float32, expect=0):
    err = err_flag()
    out = pkv.paged_decode_attn_mass(q, kp, vp, dev(bt), dev(np.asarray(lens, np.int32)), scale, mass, out_dtype=out_dtype, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == expect, int(err.item())
    return out


def check_mass(got, ref, before, q, kp, scale, lens):
    """A weight's relative error is at most twice the score's absolute one (its own and the softmax
    sum's) plus 2^-19 for the exponentials, the sum and the division; a score is an fp32 sum of d
    products: d + 8 roundings of 2^-24 of sum |q k|.  The sum with the account rounds once more."""
    d = q.shape[-1]
    big = scale * d * float(np.abs(f64(q)).max()) * float(np.abs(f64(kp)).max()) / 2
    delta = 2.0 ** -24 * (d + 8) * big
    tol = (2 * delta + 2.0 ** -19) * ref + 2.0 ** -23 * (ref + before)
    live = np.broadcast_to(np.arange(got.shape[-1]) < np.asarray(lens)[:, None, None], got.shape)
    assert np.all(np.abs(got - ref - before)[live] <= tol[live] + 1e-30)
    assert np.array_equal(got[~live], before[~live])           # behind the context: as they were
    G = q.shape[1] // got.shape[1]
    for s, n in enumerate(lens):
        if n > 0:
            assert np.allclose((got - before)[s, :, :n].sum(-1), G, rtol=1e-4, atol=1e-4 * max(1.0, n * 2.0 ** -23))


@pytest.mark.parametrize("d,bs", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 64)])
@pytest.mark.parametrize("n_h,n_kv", [(8, 8), (8, 2), (32, 8), (16, 1), (32, 1), (48, 1), (64, 1), (7, 1), (10, 2), (24, 2), (12, 1)])
def test_mass_sweep(d, bs, n_h, n_kv):
    lens = [0, 1, bs - 1, bs + 1, 3 * bs + 7, 2 * bs, 5 * bs, 70]
    kp, vp, bt, g = pools(lens, n_kv, d, bs, seed=n_h + bs)
    q = torch.randn(len(lens), n_h, d, generator=g).to(torch.bfloat16)
    T = bt.shape[1] * bs + 5                                   # rows of the accounts may be longer than the table
    mass = torch.rand(len(lens), n_kv, T, generator=g)
    scale = 1 / math.sqrt(d)
    dm, dq, dk, dv = mass.to(DEV), q.to(DEV), kp.to(DEV), vp.to(DEV)
    out = run_mass(dq, dk, dv, bt, lens, scale, dm)
    check_attention(out, oracle.paged_decode_attention(f64(q), f64(kp), f64(vp), bt, lens, scale, bs), "mass fp32")
    check_mass(f64(dm), ev.attention_mass(f64(q), f64(kp), bt, lens, scale, bs, T), f64(mass), q, kp, scale, lens)
    out16 = run_mass(dq, dk, dv, bt, lens, scale, dm, torch.bfloat16)
    check_attention(out16, oracle.paged_decode_attention(f64(q), f64(kp), f64(vp), bt, lens, scale, bs), "mass bf16")


@pytest.mark.parametrize("n_h,n_kv,lens", [(8, 2, [20000] + [3] * 300), (32, 1, [30000, 1, 0, 77]), (4, 4, [40001]), (8, 1, [9000] * 3 + [0] * 260)])
def test_mass_long_and_many(n_h, n_kv, lens):
    kp, vp, bt, g = pools(lens, n_kv, 128, 32, seed=len(lens))
    q = torch.randn(len(lens), n_h, 128, generator=g).to(torch.bfloat16)
    scale, T = 1 / math.sqrt(128), bt.shape[1] * 32
    masses = [torch.zeros(len(lens), n_kv, T, device=DEV) for _ in range(2)]
    dq, dk, dv = q.to(DEV), kp.to(DEV), vp.to(DEV)
    outs = [run_mass(dq, dk, dv, bt, lens, scale, m) for m in masses]
    assert torch.equal(outs[0], outs[1]) and torch.equal(masses[0], masses[1])
    check_attention(outs[0], oracle.paged_decode_attention(f64(q), f64(kp), f64(vp), bt, lens, scale, 32), "long")
    check_mass(f64(masses[0]), ev.attention_mass(f64(q), f64(kp), bt, lens, scale, 32, T), np.zeros(masses[0].shape), q, kp, scale, lens)


# as many units of 16 tokens per segment as change the least length of a piece; and more sequences than
# one CTA plans for
@pytest.mark.parametrize("lens", [[1008, 1024], [2032, 2048], [4080, 4096, 4096], [(7 * i) % 41 for i in range(300)]],
                         ids=["64", "128", "256", "300 sequences"])
def test_mass_piece_lengths(lens):
    kp, vp, bt, g = pools(lens, 2, 64, 16, seed=len(lens))
    q = torch.randn(len(lens), 8, 64, generator=g).to(torch.bfloat16)
    T = bt.shape[1] * 16
    mass = torch.rand(len(lens), 2, T, generator=g)
    dm, dq, dk, dv = mass.to(DEV), q.to(DEV), kp.to(DEV), vp.to(DEV)
    out = run_mass(dq, dk, dv, bt, lens, 0.125, dm)
    check_attention(out, oracle.paged_decode_attention(f64(q), f64(kp), f64(vp), bt, lens, 0.125, 16), "mass fp32")
    check_mass(f64(dm), ev.attention_mass(f64(q), f64(kp), bt, lens, 0.125, 16, T), f64(mass), q, kp, 0.125, lens)


def test_mass_stale_rows_bad_blocks_and_lengths():
    lens = [100, 64, 30, 50]
    kp, vp, bt, g = pools(lens, 2, 64, 16, seed=4)
    q = torch.randn(4, 8, 64, generator=g).to(torch.bfloat16)
    for s, n in enumerate(lens):                               # NaN and infinities behind the context
        if n % 16:
            kp[bt[s, n // 16], :, n % 16:] = float("nan")
            vp[bt[s, n // 16], :, n % 16:] = float("inf")
    ref = oracle.paged_decode_attention(f64(q), f64(kp), f64(vp), bt, lens, 0.125, 16)
    mass = torch.zeros(4, 2, bt.shape[1] * 16, device=DEV)
    ws = torch.full((pkv.mass_workspace_bytes(4, 8, 2, 64, 16, bt.shape[1]),), 255, dtype=torch.uint8, device=DEV)   # NaN scores
    err = err_flag()
    out = pkv.paged_decode_attn_mass(q.to(DEV), kp.to(DEV), vp.to(DEV), dev(bt), dev(np.array(lens, np.int32)), 0.125, mass,
                                     out_dtype=torch.float32, workspace=ws, err=err)
    check_attention(out, ref, "stale rows")
    check_mass(f64(mass), ev.attention_mass(f64(q), f64(kp), bt, lens, 0.125, 16, mass.shape[2]), np.zeros(mass.shape), q,
               torch.nan_to_num(kp, nan=0.0), 0.125, lens)
    bad = bt.copy()
    bad[0, 2], bad[1, :], bad[2, 0] = kp.shape[0], -5, 10 ** 9
    mass.zero_()
    ws.fill_(255)
    out = pkv.paged_decode_attn_mass(q.to(DEV), kp.to(DEV), vp.to(DEV), dev(bad), dev(np.array(lens, np.int32)), 0.125, mass,
                                     out_dtype=torch.float32, workspace=ws, err=err)
    assert int(err.item()) == pkv.DEV_BAD_BLOCK
    m = f64(mass)
    assert not m[1].any() and not f64(out)[1].any() and not m[0, :, 32:48].any() and not m[2, :, :16].any()
    for s, skip in ((0, [2]), (2, [0])):
        rows = [t for t in range(lens[s]) if t // 16 not in skip]
        for gk in range(2):
            k = np.stack([f64(kp)[bt[s, t // 16], gk, t % 16] for t in rows])
            w = sum(oracle.attention_weights(f64(q[s, h]), k, 0.125) for h in range(4 * gk, 4 * gk + 4))
            assert np.allclose(m[s, gk, rows], w, rtol=1e-4, atol=1e-9)
    mass.zero_()
    over = [100, 7 * 16 + 50, -4, 50]
    run_mass(q.to(DEV), kp.nan_to_num(0.0).to(DEV), vp.nan_to_num(0.0, posinf=0.0).to(DEV), np.maximum(bt, 0), over, 0.125, mass, expect=pkv.DEV_BAD_CTX)
    assert not f64(mass)[2].any() and np.isfinite(f64(mass)).all()


def test_existing_attention_with_only_bad_blocks_gives_zeros():
    # a row all of whose pieces hold bad blocks, through the split merge (narrow and wide)
    for batch in (1, 40):
        q = torch.randn(batch, 8, 64, device=DEV).to(torch.bfloat16)
        pool = torch.randn(4, 2, 16, 64, device=DEV).to(torch.bfloat16)
        bt = torch.full((batch, 600), 77, dtype=torch.int32, device=DEV)
        ctx = torch.full((batch,), 9600, dtype=torch.int32, device=DEV)
        err = err_flag()
        out = pkv.paged_decode_attn(q, pool, pool, bt, ctx, 0.125, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == pkv.DEV_BAD_BLOCK and not out.any()


# ---- eviction ---------------------------------------------------------------------------------------
def state_of(B, n_kv, T, lens, kept, rng, ties=False):
    mass = rng.exponential(size=(B, n_kv, T)).astype(np.float32)
    if ties:
        mass = np.round(mass * 2).astype(np.float32)           # many equal accounts
    dropped = rng.integers(0, 50, size=B).astype(np.int32)
    kept = np.minimum(np.asarray(kept, np.int32), np.asarray(lens, np.int32))
    pos = np.zeros((B, n_kv, T), np.int32)
    for s in range(B):
        for g in range(n_kv):                                  # distinct tokens among the first dropped + kept
            pos[s, g, :kept[s]] = rng.permutation(dropped[s] + kept[s])[:kept[s]]
    return mass, pos, kept, dropped


def run_evict(kp, vp, bt, lens, keep, recent, st, in_place, expect=0):
    dk, dv = kp.to(DEV), vp.to(DEV)
    mass, pos, kept, dropped = st
    state = pkv.EvictState(dev(mass), dev(pos), dev(kept), dev(dropped))
    out = None if in_place else pkv.EvictState(torch.full_like(state.mass, -3.0), torch.full_like(state.positions, -3),
                                               torch.full_like(state.kept, -3), torch.full_like(state.dropped, -3))
    err = err_flag()
    new = pkv.kv_evict(dk, dv, dev(bt), dev(np.asarray(lens, np.int32)), dev(np.asarray(keep, np.int32)), recent, state, out=out, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == expect
    return dk, dv, (state if in_place else out), new, state


def check_evict(kp, vp, bt, lens, keep, recent, st, bs, in_place):
    dk, dv, got, new, src = run_evict(kp, vp, bt, lens, keep, recent, st, in_place)
    mass, pos, kept, dropped = st
    wk, wv, wm, wp, wkept, wdrop, wnew = ev.evict(f64(kp), f64(vp), bt, lens, keep, recent, mass, pos, kept, dropped, bs)
    assert np.array_equal(f64(dk), wk) and np.array_equal(f64(dv), wv)
    assert np.array_equal(got.kept.cpu().numpy(), wkept) and np.array_equal(got.dropped.cpu().numpy(), wdrop)
    assert np.array_equal(new.cpu().numpy(), wnew)
    gm, gp = got.mass.cpu().numpy(), got.positions.cpu().numpy()
    for s, n in enumerate(lens):
        K = wkept[s]
        assert np.array_equal(gm[s, :, :n], wm[s, :, :n], equal_nan=True), s
        assert np.array_equal(gp[s, :, :K], wp[s, :, :K]), s
        rest_m, rest_p = (mass, pos) if in_place else (np.full_like(mass, -3), np.full_like(pos, -3))
        assert np.array_equal(gm[s, :, n:], rest_m[s, :, n:], equal_nan=True)
        assert np.array_equal(gp[s, :, K:], rest_p[s, :, K:])
    if not in_place:
        assert np.array_equal(src.mass.cpu().numpy(), mass, equal_nan=True) and np.array_equal(src.positions.cpu().numpy(), pos)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("d,bs,n_kv,recent", [(64, 16, 2, 0), (128, 16, 8, 7), (128, 32, 1, 1000), (64, 64, 3, 16), (128, 64, 2, 1)])
def test_evict_matches_oracle(d, bs, n_kv, recent, ties, in_place):
    lens = [0, 1, 5, bs, 3 * bs + 5, 200, 333, 64]
    keep = [3, 0, 5, bs - 1, bs + 3, 150, 16, 1]
    kp, vp, bt, _ = pools(lens, n_kv, d, bs, seed=d + bs)
    st = state_of(len(lens), n_kv, bt.shape[1] * bs + 3, lens, [0, 1, 2, 0, bs, 100, 333, 64], np.random.default_rng(recent), ties)
    check_evict(kp, vp, bt, lens, keep, recent, st, bs, in_place)


@pytest.mark.parametrize("batch,n_kv,n,keep,recent", [(1, 1, 40000, 10001, 500), (2, 3, 9001, 9000, 10), (1, 1, 4097, 1, 0), (40, 8, 700, 300, 50),
                                                      (1, 2, 5000, 4999, 4999)])
def test_evict_long_clusters_and_many(batch, n_kv, n, keep, recent):
    bs = 16
    lens = [max(1, n - 37 * s) for s in range(batch)]
    kp, vp, bt, _ = pools(lens, n_kv, 64, bs, seed=n)
    st = state_of(batch, n_kv, bt.shape[1] * bs, lens, [n // 3] * batch, np.random.default_rng(n))
    check_evict(kp, vp, bt, lens, [keep] * batch, recent, st, bs, True)


# every shape of the selection: threads and rows per thread, one CTA or a cluster
@pytest.mark.parametrize("batch,n_kv,n,keep", [(1, 2, 1024, 700), (3, 2, 1500, 40), (2, 2, 2048, 2047), (330, 2, 1100, 1000), (3, 2, 3000, 1700),
                                               (2, 1, 4096, 2048), (1, 2, 20000, 7000), (1, 2, 70000, 69000)])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_selection_shapes(batch, n_kv, n, keep, in_place):
    bs = 16
    lens = [max(1, n - 3 * s) for s in range(batch)]
    kp, vp, bt, _ = pools(lens, n_kv, 64, bs, seed=n)
    st = state_of(batch, n_kv, bt.shape[1] * bs, lens, [n // 3] * batch, np.random.default_rng(n), ties=n % 3 == 0)
    check_evict(kp, vp, bt, lens, [keep] * batch, 33, st, bs, in_place)


def test_evict_special_accounts():
    # NaN above infinity, both zeros, negatives, equal accounts over CTA boundaries
    bs, n = 16, 9000
    kp, vp, bt, _ = pools([n, 64], 1, 64, bs, seed=1)
    mass, pos, kept, dropped = state_of(2, 1, bt.shape[1] * bs, [n, 64], [0, 0], np.random.default_rng(2))
    mass[0, 0, :] = 0.25
    mass[1, 0, :8] = [0.0, -0.0, np.inf, np.nan, -np.inf, -1.0, 1e-40, -np.nan]
    mass[1, 0, 8:] = -2.0
    for keep in ([5000, 1], [8999, 2], [17, 5], [1, 7]):
        check_evict(kp, vp, bt, [n, 64], keep, 0, (mass, pos, kept, dropped), bs, False)


def test_evict_rows_too_long_for_shared_memory():
    # more rows than a cluster of eight holds: keys are read again in every round
    bs, n, n_kv, d = 64, 400000, 1, 64
    blocks = n // bs
    g = torch.Generator(device=DEV).manual_seed(5)
    kp = torch.randn(blocks, n_kv, bs, d, generator=g, device=DEV).to(torch.bfloat16)
    vp = kp.clone()
    bt = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)[None]
    mass = torch.rand(1, 1, n, generator=g, device=DEV)
    st = pkv.alloc_evict_state(1, n_kv, n, DEV)
    st.mass.copy_(mass)
    keep = 123457
    full = kp[bt[0].long()].transpose(0, 1).reshape(n, d).clone()
    new = pkv.kv_evict(kp, vp, bt, dev(np.array([n], np.int32)), dev(np.array([keep], np.int32)), 1000, st)
    key = mass[0, 0].clone()
    key[n - 1000:] = 2.0
    best = torch.sort(key, descending=True, stable=True).indices[:keep]
    stay = torch.zeros(n, dtype=torch.bool, device=DEV)
    stay[best] = True
    want = torch.arange(keep, device=DEV)
    want[~stay[:keep]] = keep + stay[keep:].nonzero()[:, 0]
    assert new.tolist() == [keep] and torch.equal(st.positions[0, 0, :keep].long(), want)
    assert torch.equal(kp[bt[0].long()].transpose(0, 1).reshape(n, d)[:keep], full[want])
    assert torch.equal(st.mass[0, 0, :keep], mass[0, 0, want]) and not st.mass[0, 0, keep:].any()


def test_evict_bad_block_is_flagged_and_skipped():
    bs = 16
    kp, vp, bt, _ = pools([64], 1, 64, bs, seed=1)
    st = pkv.alloc_evict_state(1, 1, 64, DEV)
    st.mass[0, 0, :32], st.mass[0, 0, 32:] = 0.0, 1.0
    bad = bt.copy()
    bad[0, 3] = 10 ** 6
    dk, dv = kp.to(DEV), vp.to(DEV)
    err = err_flag()
    pkv.kv_evict(dk, dv, dev(bad), dev(np.array([64], np.int32)), dev(np.array([32], np.int32)), 0, st, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pkv.DEV_BAD_BLOCK
    assert torch.equal(dk[bt[0, 0]].cpu(), kp[bt[0, 2]]) and torch.equal(dk[bt[0, 1]].cpu(), kp[bt[0, 1]])


def test_refusals():
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    q, bt = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    ctx = torch.ones(2, dtype=torch.int32, device=DEV)
    st, other = (pkv.alloc_evict_state(2, 2, 32, DEV) for _ in range(2))
    mixed = pkv.EvictState(st.mass, other.positions, other.kept, other.dropped)
    short = pkv.alloc_evict_state(2, 2, 31, DEV)
    for bad in (lambda: pkv.paged_decode_attn_mass(q, kp, kp, bt, ctx, 1.0, st.mass.double()), lambda: pkv.paged_decode_attn_mass(q, kp, kp, bt, ctx, 1.0, short.mass),
                lambda: pkv.paged_decode_attn_mass(q, kp, kp, bt, ctx, 1.0, st.mass[:1]), lambda: pkv.paged_decode_attn_mass(q, kp, kp, bt.long(), ctx, 1.0, st.mass),
                lambda: pkv.paged_decode_attn_mass(q, kp, kp, bt, ctx, 1.0, st.mass, workspace=torch.empty(512, dtype=torch.uint8, device=DEV)),
                lambda: pkv.mass_workspace_bytes(1, 8, 3, 64, 16, 1),
                lambda: pkv.kv_evict(kp, kp, bt, ctx, ctx, 0, short), lambda: pkv.kv_evict(kp, kp, bt, ctx, ctx.clone(), 0, st, new_lens=ctx),
                lambda: pkv.kv_evict(kp, kp, bt, ctx, ctx.clone(), 0, st, new_lens=st.kept),
                lambda: pkv.kv_evict(kp, kp, bt, ctx, ctx.clone(), -1, st), lambda: pkv.kv_evict(kp, kp, bt, ctx, ctx.clone(), 0, st, out=mixed),
                lambda: pkv.kv_evict(kp, kp, bt, ctx, ctx.long(), 0, st), lambda: pkv.kv_evict(kp.half(), kp, bt, ctx, ctx.clone(), 0, st)):
        with pytest.raises(pkv.PkvError):
            bad()


def test_graph_replays_equal_eager():
    lens, keep = [300, 77, 500], [128, 100, 33]
    kp, vp, bt, g = pools(lens, 2, 64, 16, seed=9)
    q = torch.randn(3, 8, 64, generator=g).to(torch.bfloat16).to(DEV)
    dbt, dctx, dkeep = dev(bt), dev(np.array(lens, np.int32)), dev(np.array(keep, np.int32))
    runs = []
    for graphed in (False, True):
        st = pkv.alloc_evict_state(3, 2, bt.shape[1] * 16, DEV)
        dk, dv, out, new = kp.to(DEV), vp.to(DEV), torch.empty_like(q), torch.empty_like(dctx)
        ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in
              (pkv.mass_workspace_bytes(3, 8, 2, 64, 16, bt.shape[1]), pkv.evict_workspace_bytes(3, 2, 16, bt.shape[1]))]

        def step():
            pkv.paged_decode_attn_mass(q, dk, dv, dbt, dctx, 0.125, st.mass, out=out, workspace=ws[0])
            pkv.kv_evict(dk, dv, dbt, dctx, dkeep, 20, st, new_lens=new, workspace=ws[1])
            pkv.paged_decode_attn_mass(q, dk, dv, dbt, new, 0.125, st.mass, out=out, workspace=ws[0])

        if graphed:
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                step()
            gr.replay()
        else:
            step()
        torch.cuda.synchronize()
        runs.append((out, new, dk, dv, st.mass, st.positions, st.kept, st.dropped))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


# ---- run together -----------------------------------------------------------------------------------
def test_serving_loop_with_eviction():
    """Prompts through the block manager; per step rotary append, accounted attention, and an eviction
    when a sequence passes its budget; every step against the oracle's own cache and accounts."""
    n_h, n_kv, d, bs, B, budget, recent = 8, 2, 64, 16, 3, 48, 8
    rng = np.random.default_rng(0)
    bm = pkv.BlockManager(40, bs)
    g = torch.Generator().manual_seed(0)
    kp, vp = (torch.zeros(40, n_kv, bs, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = pkv.rope_table(d, 32, interleaved=True, scaling="linear", factor=2.0)
    freqs, amp = oracle.rope_frequencies(32, scaling="linear", factor=2.0)
    seen = [37, 50, 16]
    for s in range(B):
        bm.add_sequence(s, rng.integers(0, 1000, size=seen[s]).tolist())
    mb = 8
    T = mb * bs
    st = pkv.alloc_evict_state(B, n_kv, T, DEV)
    om, op, ok, od = np.zeros((B, n_kv, T)), np.zeros((B, n_kv, T), np.int64), np.zeros(B, np.int64), np.zeros(B, np.int64)
    evictions = 0
    for step in range(30):
        if step == 0:                                          # the prompts
            bt, ctx = bm.tables(list(range(B)), mb)
            seq = np.repeat(np.arange(B), seen)
            pos = np.concatenate([np.arange(n) for n in seen])
            slots = np.concatenate([bt[s, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs for s, n in enumerate(seen)])
        else:
            slots = bm.append_tokens(list(range(B)), [1] * B)
            seq, pos = np.arange(B), np.array(seen)
            seen = [n + 1 for n in seen]
            bt, ctx = bm.tables(list(range(B)), mb)
        qkv = torch.randn(len(seq), (n_h + 2 * n_kv) * d, generator=g).to(torch.bfloat16).to(DEV)
        q, k, v = qkv.split([n_h * d, n_kv * d, n_kv * d], 1)
        q, k, v = q.view(-1, n_h, d), k.view(-1, n_kv, d), v.view(-1, n_kv, d)
        err = err_flag()
        qr = pkv.rope_append(q, k, v, dev(pos.astype(np.int32)), dev(slots), table, kp, vp, err=err)
        rk = oracle.rope_tokens(f64(k), pos, freqs, amp, True)
        got = f64(kp)[slots // bs, :, slots % bs]
        assert np.abs(got - rk).max() <= 2.0 ** -8 * np.abs(rk).max() * 1.01
        last = np.array([np.nonzero(seq == s)[0][-1] for s in range(B)])
        ql = qr[dev(last)].contiguous()
        out = pkv.paged_decode_attn_mass(ql, kp, vp, dev(bt), dev(ctx), d ** -0.5, st.mass, out_dtype=torch.float32, err=err)
        check_attention(out, oracle.paged_decode_attention(f64(ql), f64(kp), f64(vp), np.maximum(bt, 0), ctx, d ** -0.5, bs), f"step {step}")
        om += ev.attention_mass(f64(ql), f64(kp), np.maximum(bt, 0), ctx, d ** -0.5, bs, T)
        assert np.allclose(f64(st.mass), om, rtol=1e-4, atol=1e-5)
        over = [s for s in range(B) if ctx[s] >= budget + 4]
        if over:
            keep = np.array([budget if s in over else 10 ** 6 for s in range(B)], np.int32)
            # the oracle selects by the GPU's accounts: equal ones apart, fp32 and fp64 may order two of them differently
            m32 = st.mass.cpu().numpy()
            wk, wv, om, op, ok, od, wn = ev.evict(f64(kp), f64(vp), np.maximum(bt, 0), ctx, keep, recent, m32, op, ok, od, bs)
            om = om.astype(np.float64)
            new = pkv.kv_evict(kp, vp, dev(bt), dev(ctx), dev(keep), recent, st, err=err)
            for s in over:
                assert bm.evict(s, budget) == budget // bs
                evictions += 1
            assert new.tolist() == wn.tolist() == bm.tables(list(range(B)), mb)[1].tolist()
            assert np.array_equal(f64(kp), wk) and np.array_equal(f64(vp), wv)
            assert np.array_equal(st.kept.cpu().numpy(), ok) and np.array_equal(st.dropped.cpu().numpy(), od)
            for s in over:                                     # the newest tokens are all there
                for gk in range(n_kv):
                    assert set(range(seen[s] - recent, seen[s])) <= set(st.positions[s, gk, :budget].tolist())
        assert int(err.item()) == 0
    assert evictions >= 10


def test_serving_steps_over_the_8_bit_cache():
    """Rotation, quantize-on-append and attention of a prefill and decode steps, a windowed layer too."""
    n_h, n_kv, d, bs, B = 16, 4, 128, 32, 3
    lens, steps = [45, 3, 64], 5
    rng = np.random.default_rng(1)
    mb = -(-(max(lens) + steps) // bs)
    bt = rng.permutation(B * mb).reshape(B, mb).astype(np.int32)
    table = pkv.rope_table(d, base=500000.0)
    freqs, amp = oracle.rope_frequencies(d, base=500000.0)
    for fmt in ("e4m3", "int8"):
        cache = pkv.alloc_q8_cache(B * mb, n_kv, bs, d, B, fmt, DEV)
        want = oracle.Q8Cache(B * mb, n_kv, bs, d, fmt)
        n = list(lens)
        g = torch.Generator().manual_seed(5)
        for step in range(steps + 1):
            many = n if step == 0 else [1] * B
            start = [0] * B if step == 0 else n
            seq = np.repeat(np.arange(B), many)
            pos = np.concatenate([a + np.arange(b) for a, b in zip(start, many)])
            slots = bt[seq, pos // bs].astype(np.int64) * bs + pos % bs
            q, k, v = (torch.randn(len(seq), h, d, generator=g).to(torch.bfloat16).to(DEV) for h in (n_h, n_kv, n_kv))
            err = err_flag()
            qr, kr = pkv.rope_qk(q, k, dev(pos.astype(np.int32)), table)
            ref = oracle.rope_tokens(f64(k), pos, freqs, amp)
            assert np.abs(f64(kr) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() * 1.01
            pkv.kv_quant_append_q8(kr, v, dev(slots), dev(seq.astype(np.int32)), cache, err=err)
            want.append(f64(kr), f64(v), slots)
            n = n if step == 0 else [x + 1 for x in n]
            assert np.array_equal(f64(cache.k_codes.float()), want.codes[0]) and np.array_equal(cache.scales.cpu().numpy(), want.scales)
            last = np.array([np.nonzero(seq == s)[0][-1] for s in range(B)])
            ql, ctx = qr[dev(last)].contiguous(), np.array(n, np.int32)
            for window in (0, 40):
                out = pkv.paged_decode_attn_q8(ql, cache, dev(bt), dev(ctx), d ** -0.5, window=window, out_dtype=torch.float32, err=err)
                check_attention(out, oracle.paged_decode_attention(f64(ql), *want.values(), bt, ctx, d ** -0.5, bs, window=window), (fmt, step))
            assert int(err.item()) == 0
