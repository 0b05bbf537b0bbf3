"""Rotary positions of new tokens with the append, and alone, against the float64 oracle."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_175_gb300 as pkv
from gpu_common import DEV, err_flag, f64

pytestmark = pytest.mark.gpu


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy()


def close(got, ref, x, amp, what):
    """bf16's half step of the value (2^-8), and the fp32 arithmetic: the angle as a float of half turns
    (2^-24 relative of at most pi: 2^-22), sincospif (2 units: 2^-23), the amplitude, two products and a
    sum (2^-22) -- of the pair's magnitude, bounded by the row's largest pair: below 2^-20."""
    mag = amp * np.sqrt(2.0) * np.abs(x).max(axis=-1, keepdims=True)
    d = np.abs(got - ref)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * mag
    assert (d <= tol).all(), (what, float((d / tol).max()))


def case(n, n_h, n_kv, d, bs, seed, far=100000, extra_blocks=2):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    qkv = torch.randn(n, (n_h + 2 * n_kv) * d, generator=g).to(torch.bfloat16)
    blocks = -(-n // bs) + extra_blocks
    kp, vp = (torch.randn(blocks, n_kv, bs, d, generator=g).to(torch.bfloat16) for _ in range(2))
    pos = rng.integers(0, far, size=n).astype(np.int32)
    slots = rng.choice(blocks * bs, size=n, replace=False).astype(np.int64)
    return qkv, kp, vp, pos, slots


def parts(qkv, n_h, n_kv, d):
    n = qkv.shape[0]
    q, k, v = qkv.split([n_h * d, n_kv * d, n_kv * d], 1)
    return q.view(n, n_h, d), k.view(n, n_kv, d), v.view(n, n_kv, d)


def check(qkv, kp, vp, pos, slots, n_h, n_kv, d, table, freqs, amp, inter, bs, q_out=None, expect_err=0, stream=None):
    dq, dkp, dvp = qkv.to(DEV), kp.to(DEV), vp.to(DEV)
    q, k, v = parts(dq, n_h, n_kv, d)
    err = err_flag()
    out = torch.full((qkv.shape[0], n_h, d), 7.0, dtype=torch.bfloat16, device=DEV) if q_out is None else q
    got = pkv.rope_append(q, k, v, torch.as_tensor(pos, device=DEV), torch.as_tensor(slots, device=DEV), table, dkp, dvp,
                          q_out=out, err=err, stream=stream)
    torch.cuda.synchronize()
    assert int(err.item()) == expect_err
    hq, hk, hv = (f64(x) for x in parts(qkv, n_h, n_kv, d))
    live = (slots >= 0) & (slots < kp.shape[0] * bs)
    rq, rk = oracle.rope_tokens(hq, pos, freqs, amp, inter), oracle.rope_tokens(hk, pos, freqs, amp, inter)
    close(f64(got)[live], rq[live], hq[live], amp, "q")
    if (~live).any():
        want = f64(parts(qkv, n_h, n_kv, d)[0]) if q_out is not None else np.full(rq.shape, 7.0)
        assert np.array_equal(f64(got)[~live], want[~live])
    s = np.where(live, slots, -1)
    ek, ev = oracle.kv_append(f64(kp), f64(vp), rk, hv, s, bs)
    mag_src, _ = oracle.kv_append(f64(kp), f64(vp), hk, hv, s, bs)
    close(f64(dkp), ek, mag_src, amp, "k")
    assert np.array_equal(f64(dvp), ev)
    r = 2 * len(freqs)                                          # copied channels: bit for bit
    assert np.array_equal(bits(got[..., r:])[live], bits(parts(qkv, n_h, n_kv, d)[0][..., r:])[live])
    written = np.zeros(kp.shape[0] * bs, bool)
    written[slots[live]] = True
    untouched = ~written.reshape(kp.shape[0], bs)
    assert np.array_equal(bits(dkp).transpose(0, 2, 1, 3)[untouched], bits(kp).transpose(0, 2, 1, 3)[untouched])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,r,n_h,n_kv,bs,n", [(64, 64, 8, 2, 16, 1), (128, 128, 32, 8, 16, 33), (128, 32, 5, 5, 32, 100),
                                               (64, 48, 7, 1, 64, 301), (64, 16, 1, 1, 16, 700), (128, 96, 64, 1, 16, 90),
                                               (128, 128, 1, 1, 64, 513)])
def test_layouts_and_parts(d, r, n_h, n_kv, bs, n, inter):
    qkv, kp, vp, pos, slots = case(n, n_h, n_kv, d, bs, seed=n + r)
    freqs, amp = oracle.rope_frequencies(r)
    check(qkv, kp, vp, pos, slots, n_h, n_kv, d, pkv.rope_table(d, r, interleaved=inter), freqs, amp, inter, bs)


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                        ("parts", dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0)),
                                        ("yarn", dict(factor=16.0, original_len=4096.0))])
def test_scalings(scaling, kw):
    qkv, kp, vp, pos, slots = case(77, 8, 2, 128, 16, seed=5)
    freqs, amp = oracle.rope_frequencies(64, scaling=scaling, **kw)
    check(qkv, kp, vp, pos, slots, 8, 2, 128, pkv.rope_table(128, 64, scaling=scaling, **kw), freqs, amp, False, 16)


def test_far_and_negative_positions():
    qkv, kp, vp, pos, slots = case(64, 4, 2, 64, 16, seed=9)
    pos[:] = np.random.default_rng(1).integers(-2 ** 31, 2 ** 31, size=64)
    pos[:6] = [0, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 1]
    # the oracle's float64 angle is off by 2^31 * 2^-53 turns at most here, far below 2^-20
    freqs, amp = oracle.rope_frequencies(64)
    check(qkv, kp, vp, pos, slots, 4, 2, 64, pkv.rope_table(64), freqs, amp, False, 16)


def test_large_call_uses_several_items_per_thread():
    n, n_h, n_kv, d = 1700, 32, 8, 128                          # more than two CTAs per SM of four items a thread
    qkv, kp, vp, pos, slots = case(n, n_h, n_kv, d, 16, seed=3)
    dq, dkp, dvp = qkv.to(DEV), kp.to(DEV), vp.to(DEV)
    q, k, v = parts(dq, n_h, n_kv, d)
    t = pkv.rope_table(d, 64, interleaved=True)
    out = pkv.rope_append(q, k, v, torch.as_tensor(pos, device=DEV), torch.as_tensor(slots, device=DEV), t, dkp, dvp)
    # the same tokens in small calls give the same bits
    small, k2, v2 = torch.empty_like(out), kp.to(DEV), vp.to(DEV)
    for i in range(0, n, 97):
        j = min(n, i + 97)
        pkv.rope_append(q[i:j], k[i:j], v[i:j], torch.as_tensor(pos[i:j], device=DEV), torch.as_tensor(slots[i:j], device=DEV),
                        t, k2, v2, q_out=small[i:j])
    torch.cuda.synchronize()
    assert torch.equal(out, small) and torch.equal(dkp, k2) and torch.equal(dvp, v2)
    pick = np.array([0, 1, 850, 1699])
    freqs, amp = oracle.rope_frequencies(64)
    hq = f64(parts(qkv, n_h, n_kv, d)[0][pick])
    close(f64(out)[pick], oracle.rope_tokens(hq, pos[pick], freqs, amp, True), hq, amp, "sampled")


@pytest.mark.parametrize("in_place", [False, True])
def test_padding_and_bad_slots_are_left(in_place):
    qkv, kp, vp, pos, slots = case(40, 8, 2, 64, 16, seed=11)
    slots[[0, 7, 39]] = -1
    slots[[3, 20]] = kp.shape[0] * 16 + 5
    freqs, amp = oracle.rope_frequencies(32)
    check(qkv, kp, vp, pos, slots, 8, 2, 64, pkv.rope_table(64, 32), freqs, amp, False, 16,
          q_out="in place" if in_place else None, expect_err=pkv.DEV_BAD_SLOT)


def test_rope_qk_equals_rope_append_and_runs_in_place():
    n, n_h, n_kv, d = 130, 8, 2, 128
    qkv, kp, vp, pos, slots = case(n, n_h, n_kv, d, 16, seed=21)
    t = pkv.rope_table(d, 96, scaling="yarn", factor=4.0, original_len=2048.0)
    dq, dkp, dvp = qkv.to(DEV), kp.to(DEV), vp.to(DEV)
    q, k, v = parts(dq, n_h, n_kv, d)
    p = torch.as_tensor(pos, device=DEV)
    sl = torch.as_tensor(slots, device=DEV)
    a = pkv.rope_append(q, k, v, p, sl, t, dkp, dvp)
    b, kb = pkv.rope_qk(q, k, p, t)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(kb, dkp[sl // 16, :, sl % 16])
    v0 = v.clone()
    pkv.rope_qk(q, k, p, t, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, a) and torch.equal(k, kb) and torch.equal(v, v0)


def test_side_stream_and_graph():
    n, n_h, n_kv, d = 64, 8, 2, 64
    qkv, kp, vp, pos, slots = case(n, n_h, n_kv, d, 16, seed=31)
    freqs, amp = oracle.rope_frequencies(64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    check(qkv, kp, vp, pos, slots, n_h, n_kv, d, pkv.rope_table(d), freqs, amp, False, 16, stream=None)
    with torch.cuda.stream(st):
        check(qkv, kp, vp, pos, slots, n_h, n_kv, d, pkv.rope_table(d), freqs, amp, False, 16)
    torch.cuda.synchronize()
    q, k, v = parts(qkv.to(DEV), n_h, n_kv, d)
    p, sl = torch.as_tensor(pos, device=DEV), torch.as_tensor(slots, device=DEV)
    pools = [(kp.to(DEV), vp.to(DEV)) for _ in range(2)]
    eager = pkv.rope_append(q, k, v, p, sl, pkv.rope_table(d), *pools[0])
    out = torch.empty_like(eager)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.rope_append(q, k, v, p, sl, pkv.rope_table(d), *pools[1], q_out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager) and torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])


def test_refusals():
    q, k = torch.zeros(4, 8, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    p, s = torch.zeros(4, dtype=torch.int32, device=DEV), torch.arange(4, device=DEV)
    t = pkv.rope_table(64)
    ok = dict(q=q, k=k, v=k, positions=p, slot_mapping=s, table=t, k_pool=pool, v_pool=pool.clone())
    pkv.rope_append(**ok)
    wide = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(table=pkv.rope_table(128)), dict(positions=p.long()), dict(slot_mapping=s.int()), dict(q=q.float()),
                dict(q=wide[..., ::2]), dict(positions=p[:3]), dict(k=k[:3]), dict(q=wide), dict(q_out=q[:3]),
                dict(v_pool=pool[:, :, :8]), dict(q=torch.zeros(4, 8 * 64 + 4, dtype=torch.bfloat16, device=DEV)[:, :512].view(4, 8, 64)),
                dict(k=torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV).expand(4, 2, 64))):
        with pytest.raises(pkv.PkvError):
            pkv.rope_append(**{**ok, **bad})
    empty = pkv.rope_append(q[:0], k[:0], k[:0], p[:0], s[:0], t, pool, pool)
    assert empty.shape == (0, 8, 64)
