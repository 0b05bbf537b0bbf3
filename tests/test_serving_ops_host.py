"""Host side of the rotary, 8-bit and eviction operators: the angle tables, the oracles' pins, the
block manager's eviction against its oracle, and the bindings' refusals.  No GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_175_gb300 as pkv
from oracle import evict as ev
from paged_kv_cache_175_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_library()


SCALINGS = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
            ("parts", dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0)),
            ("yarn", dict(factor=16.0, original_len=4096.0))]


@pytest.mark.parametrize("scaling,kw", SCALINGS)
@pytest.mark.parametrize("d,r", [(64, 64), (128, 128), (128, 32), (64, 48), (64, 16)])
def test_rope_table_holds_the_frequencies(scaling, kw, d, r):
    t = pkv.rope_table(d, r, base=500000.0, scaling=scaling, **kw)
    freqs, amp = oracle.rope_frequencies(r, base=500000.0, scaling=scaling, **kw)
    got = np.array(list(t.turns)[:r // 2], dtype=np.float64) * 2.0 ** -64 * 2 * math.pi
    # float64 pow and log on both sides: a few units of 2^-52, and the 2^-64 step of the table
    assert np.all(np.abs(got - freqs) <= 2.0 ** -46 * freqs + 2.0 ** -61)
    assert abs(t.amplitude - amp) <= 2.0 ** -24 * amp
    assert list(t.turns)[r // 2:] == [0] * (64 - r // 2)


def test_rope_frequencies_limits():
    # no stretch: every scaling is the plain embedding; the first pair turns by 1 per position
    f0, _ = oracle.rope_frequencies(64)
    assert f0[0] == 1.0 and abs(f0[-1] - 10000.0 ** (-62 / 64)) < 1e-12
    for scaling, kw in SCALINGS[1:]:
        f, a = oracle.rope_frequencies(64, scaling=scaling, **dict(kw, factor=1.0))
        assert np.allclose(f, f0, rtol=1e-14) and a == 1.0
    # parts and yarn: fast pairs untouched, slow pairs divided
    for scaling, kw in SCALINGS[3:]:
        f, _ = oracle.rope_frequencies(64, scaling=scaling, **kw)
        assert f[0] == f0[0] and abs(f[-1] * kw["factor"] / f0[-1] - 1) < 1e-12


def test_rope_tokens_keeps_norms_and_relative_angles():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(2, 1, 64))
    f, _ = oracle.rope_frequencies(32)
    for inter in (False, True):
        a, b = oracle.rope_tokens(x, [10, 3], f, interleaved=inter), oracle.rope_tokens(x, [1010, 1003], f, interleaved=inter)
        assert np.allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.allclose((a[0] * a[1]).sum(), (b[0] * b[1]).sum())
        assert np.array_equal(a[..., 32:], x[..., 32:])


@pytest.mark.parametrize("bad", [dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=192), dict(base=1.0),
                                 dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=2.0),
                                 dict(scaling="parts", factor=2.0, original_len=100.0, low=4.0, high=4.0)])
def test_rope_table_refusals(bad):
    with pytest.raises(pkv.PkvError):
        pkv.rope_table(128, **bad)
    with pytest.raises(pkv.PkvError):
        pkv.rope_table(96)
    with pytest.raises(ValueError):
        pkv.rope_table(128, scaling="other")


def test_round_e4m3_matches_torch_on_every_code_and_tie():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    codes = np.unique(codes[np.isfinite(codes)])
    mid = (codes[1:] + codes[:-1]) / 2
    x = np.concatenate([codes, mid, np.nextafter(mid, 1e9), np.nextafter(mid, -1e9), [460.0, 1e6, -1e6]])
    x = np.unique(x.astype(np.float32)).astype(np.float64)
    t = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.round_e4m3(x), t)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_quantize_rows_error_is_half_a_step(fmt):
    x = oracle.round_bf16(np.random.default_rng(1).normal(size=(16, 64)) * 3)
    c, s = oracle.quantize_rows(x, fmt)
    held = c * float(s)
    big = np.abs(x).max()
    # int8: half a unit of big / 127; e4m3: 2^-4 of the value, or half the subnormal step 2^-9
    step = big / 127 / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * float(s))
    # and five float32 roundings of the value: 1 / big, its product with M and x * inv move the point
    # that is rounded by |x| 2^-24 each (in units of the value), 1 / M and its product with big the
    # value held by as much
    tol = step + np.abs(x) * (5 * 2.0 ** -24 * (1 + 1e-6))
    assert np.all(np.abs(held - x) <= tol) and np.abs(held).max() >= big * (1 - 1e-6)
    z, s0 = oracle.quantize_rows(np.full((4, 4), 2.0 ** -111), fmt)
    assert s0 == 0 and not z.any()


def test_record_views_are_the_documented_order():
    bs, d = 32, 64
    c = pkv.Q8CacheTensors(torch.zeros(1, 1, 2 * bs * d + 16, dtype=torch.uint8), torch.zeros(1, 1, bs, d, dtype=torch.bfloat16),
                           torch.zeros(1, 1, bs, d, dtype=torch.bfloat16), "int8")
    rng = np.random.default_rng(2)
    want = rng.integers(-127, 128, size=(2, bs, d)).astype(np.int8)
    rec = c.records.numpy()[0, 0]
    for t in range(bs):
        for ch in range(d):
            # K: token 8 b + i, channel 16 a + 8 c + 2 j + e; V: token 8 c + 2 j + e, channel 16 a + 8 b + i
            base = (t // 16) * 16 * d + (ch // 32) * 512
            x, y = t % 16, ch % 32
            k = base + (4 * (x % 8) + (y % 8) // 2) * 16 + 8 * (y // 16) + 4 * (x // 8) + 2 * ((y % 16) // 8) + y % 2
            v = base + (4 * (y % 8) + (x % 8) // 2) * 16 + 8 * (y // 16) + 4 * ((y % 16) // 8) + 2 * (x // 8) + x % 2
            rec[k], rec[bs * d + v] = want[0, t, ch].view(np.uint8), want[1, t, ch].view(np.uint8)
    assert np.array_equal(c.k_codes[0, 0].numpy(), want[0]) and np.array_equal(c.v_codes[0, 0].numpy(), want[1])
    assert pkv.q8_record_bytes(bs, d) == 2 * bs * d + 16 and pkv.q8_record_bytes(8, 64) == 0


def test_attention_mass_sums_to_the_group():
    rng = np.random.default_rng(3)
    q, k = rng.normal(size=(3, 6, 16)), rng.normal(size=(9, 2, 4, 16))
    m = ev.attention_mass(q, k, np.arange(9).reshape(3, 3), [0, 5, 12], 0.25, 4, 12)
    assert np.allclose(m.sum(-1), [[0, 0], [3, 3], [3, 3]]) and not m[1, :, 5:].any()


def test_evict_rows_rules():
    m = np.array([5.0, 1.0, 1.0, 9.0, 2.0, 2.0, 0.5, 0.1])
    pos = np.arange(8)
    assert ev.evict_rows(m, pos, 8, 8, 0, 8) == ([], [])
    assert ev.evict_rows(m, pos, 8, 4, 2, 8) == ([1, 2], [6, 7])       # the two newest, then 9 and 5
    assert ev.evict_rows(m, pos, 8, 3, 0, 8) == ([1, 2], [3, 4])       # of the equal twos the lower row
    assert ev.evict_rows(m, pos, 8, 2, 100, 8) == ([0, 1], [6, 7])     # recent is cut to the budget
    assert ev.evict_rows(m, pos[::-1], 8, 2, 1, 8) == ([1], [3])       # newest is row 0
    assert ev.evict_rows(m, pos, 8, 2, 1, 9) == ([1], [3])             # the newest token was evicted before
    n = m.copy()
    n[6] = np.nan
    assert ev.evict_rows(n, pos, 8, 1, 0, 8) == ([0], [6])             # NaN above everything


@pytest.mark.parametrize("seed", range(6))
def test_block_manager_evict_matches_oracle(seed):
    rng = np.random.default_rng(seed)
    bs, N = 4, 60
    a, b = pkv.BlockManager(N, bs, 8), oracle.BlockManager(N, bs, 8)
    live, prompts, nxt, evicted = [], [rng.integers(0, 3, size=40).tolist() for _ in range(4)], 0, 0
    for _ in range(400):
        op = rng.integers(0, 5)
        if op == 0 and len(live) < 5:
            toks = prompts[rng.integers(4)][:rng.integers(1, 40)]
            try:
                want = b.add_sequence(nxt, toks)
            except oracle.OutOfBlocks:
                with pytest.raises(pkv.PkvError):
                    a.add_sequence(nxt, toks)
            else:
                assert a.add_sequence(nxt, toks) == (want[0], want[1])
                live.append(nxt)
            nxt += 1
        elif op == 1 and live:
            i = live.pop(rng.integers(len(live)))
            a.release(i)
            b.release(i)
        elif op in (2, 3) and live:
            i = live[rng.integers(len(live))]
            try:
                want = b.append_token(i, 1)
            except oracle.OutOfBlocks:
                with pytest.raises(pkv.PkvError):
                    a.append_tokens([i], [1])
            else:
                assert a.append_tokens([i], [1]).tolist() == [want]
        elif op == 4 and live:
            i = live[rng.integers(len(live))]
            keep = int(rng.integers(0, 30))
            try:
                want = b.evict(i, keep)
            except ValueError:
                with pytest.raises(pkv.PkvError):
                    a.evict(i, keep)
            else:
                assert a.evict(i, keep) == want
                evicted += 1
        for i in live:
            t, c = a.tables([i], 40)
            wt, wc = b.table(i)
            assert c[0] == wc and t[0][:len(wt)].tolist() == wt and (t[0][len(wt):] == -1).all()
        assert [tuple(x) for x in a.take_copies().tolist()] == b.take_copies()
        ca = a.counts()
        assert all(ca[k] == v for k, v in b.counts().items())
    assert evicted > 5


def test_block_manager_evict_refuses_shared_and_unknown():
    bm = pkv.BlockManager(32, 4)
    bm.add_sequence(1, list(range(12)))
    _, reused = bm.add_sequence(2, list(range(12)) + [7, 8, 9])
    assert reused > 0
    for seq, keep in ((2, 8), (9, 3), (2, 0), (2, 99)):
        with pytest.raises(pkv.PkvError):
            bm.evict(seq, keep)
    assert bm.evict(2, 15) == 4                                       # its whole length: nothing changes
    bm.release(1)
    assert bm.evict(2, 8) == 2                                        # alone now; its prefix leaves the tree
    assert bm.add_sequence(3, list(range(12)))[1] == 0


def test_bindings_refuse_cpu_tensors():
    z = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    pool = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    i32, i64 = torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    t = pkv.rope_table(64)
    c = pkv.alloc_q8_cache(1, 1, 16, 64, 1, device="cpu")
    st = pkv.alloc_evict_state(1, 1, 16, device="cpu")
    for call in (lambda: pkv.rope_append(z, z, z, i32, i64, t, pool, pool), lambda: pkv.rope_qk(z, z, i32, t),
                 lambda: pkv.kv_quant_append_q8(z, z, i64, i32, c),
                 lambda: pkv.paged_decode_attn_q8(z, c, i32[None], i32, 1.0),
                 lambda: pkv.paged_decode_attn_mass(z, pool, pool, i32[None], i32, 1.0, st.mass),
                 lambda: pkv.kv_evict(pool, pool, i32[None], i32, i32, 0, st)):
        with pytest.raises(pkv.PkvError):
            call()
    for table in (None, 0, ctypes.create_string_buffer(64)):            # not a table: never read as one
        with pytest.raises(pkv.PkvError):
            pkv.rope_append(z, z, z, i32, i64, table, pool, pool)
        with pytest.raises(pkv.PkvError):
            pkv.rope_qk(z, z, i32, table)
    with pytest.raises(ValueError):
        pkv.alloc_q8_cache(1, 1, 16, 96, 1, device="cpu")


def test_c_entries_refuse_bad_arguments():
    """Status codes before anything is launched (null or misaligned pointers, shapes, strides)."""
    L = pkv.lib()
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 255) & ~255
    t = pkv.rope_table(64)
    tp = ctypes.addressof(t)
    rope = lambda **k: L.pkv_rope_append(*[{**dict(q=p, qs=512, k=p, ks=128, v=p, vs=128, pos=p, slot=p, n=1, t=tp, qo=p, qos=512,
                                                   kp=p, vp=p, nb=4, bs=16, nh=8, nkv=2, d=64, e=None, s=None), **k}[x] for x in
                                            "q qs k ks v vs pos slot n t qo qos kp vp nb bs nh nkv d e s".split()])
    assert rope(n=0) == 0
    for bad in (dict(n=-1), dict(d=128), dict(d=96), dict(bs=8), dict(t=None), dict(q=None), dict(q=p + 2), dict(qs=511), dict(qs=256),
                dict(ks=129), dict(slot=None), dict(nh=0)):
        assert rope(**bad) == -1, bad
    q8 = lambda **k: L.pkv_kv_quant_append_q8(*[{**dict(k=p, ks=128, v=p, vs=128, slot=p, ts=p, n=1, f=0, c=p, kt=p, vt=p, tr=1, nb=4,
                                                        bs=16, nkv=2, d=64, e=None, s=None), **k}[x] for x in
                                                 "k ks v vs slot ts n f c kt vt tr nb bs nkv d e s".split()])
    assert q8(n=0) == 0 and q8(n=0x7fff0001) == -2
    for bad in (dict(n=-1), dict(f=2), dict(bs=128), dict(d=80), dict(ks=64), dict(vs=132), dict(c=p + 8), dict(vt=None), dict(tr=-1)):
        assert q8(**bad) == -1, bad
    ev_ = lambda **k: L.pkv_kv_evict(*[{**dict(kp=p, vp=p, bt=p, mb=2, ctx=p, keep=p, rec=0, m=p, pos=p, kd=p, dr=p, mo=p, po=p, ko=p,
                                              do=p, st=32, nl=p + 256, b=1, nkv=1, d=64, bs=16, nb=4, ws=p, wb=1 << 20, e=None, s=None),
                                         **k}[x] for x in
                                       "kp vp bt mb ctx keep rec m pos kd dr mo po ko do st nl b nkv d bs nb ws wb e s".split()])
    assert ev_(b=0) == 0
    for bad in (dict(nl=p), dict(mo=p + 512), dict(st=31), dict(rec=-1), dict(d=32), dict(bs=48), dict(ws=p + 16), dict(nl=None)):
        assert ev_(**bad) == -1, bad
    assert ev_(wb=16) == -4
    assert ev_(mb=0x7fff001, st=0x7fff0010) == -2 and L.pkv_evict_workspace_bytes(1, 1, 16, 0x7fff001) == 0
    att = lambda **k: L.pkv_paged_decode_attn_q8(*[{**dict(q=p, c=p, f=0, bt=p, mb=2, ctx=p, sc=1.0, w=0, b=1, nh=2, nkv=1, d=64, bs=16, nb=4,
                                                           o=p, ot=0, ws=p, wb=0, e=None, s=None), **k}[x] for x in
                                                    "q c f bt mb ctx sc w b nh nkv d bs nb o ot ws wb e s".split()])
    mas = lambda **k: L.pkv_paged_decode_attn_mass(*[{**dict(q=p, k=p, v=p, bt=p, mb=2, ctx=p, sc=1.0, b=1, nh=2, nkv=1, d=64, bs=16, nb=4,
                                                             o=p, ot=0, m=p, st=32, ws=p, wb=0, e=None, s=None), **k}[x] for x in
                                                      "q k v bt mb ctx sc b nh nkv d bs nb o ot m st ws wb e s".split()])
    assert att(b=0) == mas(b=0) == 0
    assert att(mb=0x7fff001) == mas(mb=0x7fff001, st=0x7fff0010) == -2 and L.pkv_mass_workspace_bytes(1, 1, 1, 64, 16, 0x7fff001) == 0
    for bad in (dict(d=96), dict(bs=8), dict(nh=65), dict(q=None), dict(o=p + 2), dict(ot=2), dict(ctx=None)):
        assert att(**bad) == mas(**bad) == -1, bad
    assert att(w=-1) == att(f=2) == mas(st=31) == -1
    assert L.pkv_evict_workspace_bytes(2, 3, 16, 10) > 0 and L.pkv_evict_workspace_bytes(2, 3, 24, 10) == 0
    assert L.pkv_q8_workspace_bytes(1, 6, 4, 64, 16, 0) == 0 and L.pkv_mass_workspace_bytes(1, 65, 1, 64, 16, 4) == 0
