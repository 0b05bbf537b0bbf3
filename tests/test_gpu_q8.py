"""The 8-bit cache: quantize-on-append bit for bit, and attention over the values held."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_175_gb300 as pkv
from gpu_common import BAR_F32_MAXABS, DEV, check_attention, err_flag, f64

pytestmark = pytest.mark.gpu


def tables(lens, bs, rng, spare=3):
    nb = [-(-int(n) // bs) for n in lens]
    blocks = sum(nb) + spare
    perm = rng.permutation(blocks).astype(np.int32)
    bt = np.full((len(lens), max(max(nb), 1)), -1, np.int32)
    cur = 0
    for s, n in enumerate(nb):
        bt[s, :n] = perm[cur:cur + n]
        cur += n
    return bt, blocks


def slots_of(bt, s, lo, hi, bs):
    r = np.arange(lo, hi)
    return bt[s, r // bs].astype(np.int64) * bs + r % bs


def dev(x):
    return torch.as_tensor(x, device=DEV)


def assert_cache(cache, ref, blocks, what=""):
    """Codes and scales of the listed blocks, bit for bit (a zero's sign aside)."""
    assert np.array_equal(f64(cache.k_codes.float())[blocks], ref.codes[0][blocks]), what
    assert np.array_equal(f64(cache.v_codes.float())[blocks], ref.codes[1][blocks]), what
    assert np.array_equal(cache.scales.cpu().numpy()[blocks], ref.scales[blocks]), what


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,bs,n_kv", [(64, 16, 2), (128, 16, 8), (128, 32, 1), (64, 64, 5), (128, 64, 2)])
def test_append_is_bit_exact_in_any_chunks(fmt, d, bs, n_kv):
    rng = np.random.default_rng(d + bs)
    lens = [1, bs, bs + 1, 3 * bs + 7, 2 * bs - 1, 5]
    bt, blocks = tables(lens, bs, rng)
    g = torch.Generator().manual_seed(3)
    ks = [(torch.randn(n, n_kv, d, generator=g) * 3).to(torch.bfloat16) for n in lens]
    vs = [torch.randn(n, n_kv, d, generator=g).to(torch.bfloat16) for n in lens]
    want = oracle.Q8Cache(blocks, n_kv, bs, d, fmt)
    for s, n in enumerate(lens):
        want.append(f64(ks[s]), f64(vs[s]), slots_of(bt, s, 0, n, bs))
    used = np.concatenate([bt[s, :-(-n // bs)] for s, n in enumerate(lens)])

    def run(cuts):
        """cuts: for each call, the [lo, hi) of each sequence."""
        cache = pkv.alloc_q8_cache(blocks, n_kv, bs, d, len(lens), fmt, DEV)
        for call in cuts:
            k = torch.cat([ks[s][a:b] for s, (a, b) in enumerate(call)])
            v = torch.cat([vs[s][a:b] for s, (a, b) in enumerate(call)])
            sl = np.concatenate([slots_of(bt, s, a, b, bs) for s, (a, b) in enumerate(call)])
            ts = np.concatenate([np.full(b - a, s, np.int32) for s, (a, b) in enumerate(call)])
            err = err_flag()
            pkv.kv_quant_append_q8(k.to(DEV), v.to(DEV), dev(sl), dev(ts), cache, err=err)
            assert int(err.item()) == 0
        return cache

    whole = run([[(0, n) for n in lens]])
    assert_cache(whole, want, used, "one call")
    tokens = run([[(min(i, n), min(i + 1, n)) for n in lens] for i in range(max(lens))])
    assert torch.equal(tokens.records, whole.records)
    # chunks that begin and end inside blocks, some running over whole blocks: the tail is read for
    # the first block and written for the last in the same call
    step = bs // 2 + 3
    chunks = run([[(min(i, n), min(i + (step if j % 2 else 2 * bs + 1), n)) for n in lens]
                  for j, i in ((0, 0), (1, 2 * bs + 1), (0, 2 * bs + 1 + step), (0, 4 * bs + 2 + step))])
    assert torch.equal(chunks.records, whole.records)
    cut = run([[(0, n // 2) for n in lens], [(n // 2, n) for n in lens]])
    assert torch.equal(cut.records, whole.records)
    for c in (whole, tokens, chunks, cut):                     # open rows are in the tails
        for s, n in enumerate(lens):
            if n % bs:
                assert torch.equal(c.k_tail[s, :, :n % bs].cpu(), ks[s][n - n % bs:].transpose(0, 1))
                assert torch.equal(c.v_tail[s, :, :n % bs].cpu(), vs[s][n - n % bs:].transpose(0, 1))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_long_call_uses_spans(fmt):
    # above the number of tokens from which a CTA takes a block_size span of them
    d, bs, n_kv = 64, 32, 3
    rng = np.random.default_rng(8)
    lens = [1500, 7, 900, 33, 64]
    start = [5, 31, 0, 32, 1]
    bt, blocks = tables(lens, bs, rng)
    g = torch.Generator().manual_seed(4)
    ks = [torch.randn(n, n_kv, d, generator=g).to(torch.bfloat16) for n in lens]
    vs = [torch.randn(n, n_kv, d, generator=g).to(torch.bfloat16) for n in lens]
    caches = [pkv.alloc_q8_cache(blocks, n_kv, bs, d, len(lens), fmt, DEV) for _ in range(2)]
    kk, vv, sl, ts = [], [], [], []
    for s, n in enumerate(lens):
        a = min(start[s], n)
        first = (ks[s][:a].to(DEV), vs[s][:a].to(DEV), dev(slots_of(bt, s, 0, a, bs)), torch.full((a,), s, dtype=torch.int32, device=DEV))
        for c in caches:
            pkv.kv_quant_append_q8(*first, c)
        kk.append(ks[s][a:]); vv.append(vs[s][a:]); sl.append(slots_of(bt, s, a, n, bs)); ts.append(np.full(n - a, s, np.int32))
    pad = 17                                                    # padding behind the last sequence
    kk.append(torch.ones(pad, n_kv, d, dtype=torch.bfloat16)); vv.append(kk[-1]); sl.append(np.full(pad, -1, np.int64)); ts.append(np.zeros(pad, np.int32))
    assert sum(len(x) for x in sl) > 2048
    err = err_flag()
    pkv.kv_quant_append_q8(torch.cat(kk).to(DEV), torch.cat(vv).to(DEV), dev(np.concatenate(sl)), dev(np.concatenate(ts)), caches[0], err=err)
    assert int(err.item()) == 0
    for x in zip(kk[:-1], vv[:-1], sl, ts):                     # a sequence per call: one token a span
        pkv.kv_quant_append_q8(x[0].to(DEV), x[1].to(DEV), dev(x[2]), dev(x[3]), caches[1])
    assert torch.equal(caches[0].records, caches[1].records)
    for s, n in enumerate(lens):
        if n % bs:
            for i, src in enumerate((ks, vs)):
                for c in caches:
                    tail = (c.k_tail, c.v_tail)[i]
                    assert torch.equal(tail[s, :, :n % bs].cpu(), src[s][n - n % bs:].transpose(0, 1))
    want = oracle.Q8Cache(blocks, n_kv, bs, d, fmt)
    want.append(f64(ks[2]), f64(vs[2]), slots_of(bt, 2, 0, lens[2], bs))
    assert_cache(caches[0], want, bt[2, :-(-lens[2] // bs)])


def test_append_after_a_cut_inside_the_open_block():
    # rows taken back from the unfinished block are overwritten: the record is that of the rows that remain
    d, bs, n_kv = 64, 16, 2
    k, v = (torch.randn(30, n_kv, d, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) for i in (1, 2))
    caches = [pkv.alloc_q8_cache(3, n_kv, bs, d, 1, "e4m3", DEV) for _ in range(2)]
    seq = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)
    put = lambda c, x, y, lo: pkv.kv_quant_append_q8(x.to(DEV), y.to(DEV), torch.arange(lo, lo + len(x), device=DEV), seq(len(x)), c)
    put(caches[0], k[:27], v[:27], 0)
    put(caches[0], k[27:], v[27:], 20)                          # rows 20..26 taken back
    put(caches[1], torch.cat([k[:20], k[27:]]), torch.cat([v[:20], v[27:]]), 0)
    assert torch.equal(caches[0].records, caches[1].records)


def test_append_strided_padding_bad_slots_and_extremes():
    d, bs, n_kv = 64, 16, 2
    cache = pkv.alloc_q8_cache(6, n_kv, bs, d, 2, "e4m3", DEV)
    before = torch.full_like(cache.records, 99)
    cache.records.copy_(before)
    cache.k_tail.fill_(5.0)
    kv = torch.randn(6, 2 * n_kv * d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    kv[0] = 0.0                                                # an all-zero row alone in its block
    kv[1] = 2.0 ** -115                                        # below the smallest scale that is kept
    kv[2, :3] = torch.tensor([3e38, -3e38, 1e-30])
    k, v = kv[:, :n_kv * d].view(6, n_kv, d), kv[:, n_kv * d:].view(6, n_kv, d)
    dk = kv.to(DEV)
    sl = np.array([0 * 16, 1 * 16, 2 * 16, -1, 6 * 16, 3 * 16], np.int64)
    ts = np.array([0, 1, 0, 0, 1, 7], np.int32)                # the last one's tail row is out of range
    err = err_flag()
    pkv.kv_quant_append_q8(dk[:, :n_kv * d].view(6, n_kv, d), dk[:, n_kv * d:].view(6, n_kv, d), dev(sl), dev(ts), cache, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pkv.DEV_BAD_SLOT
    want = oracle.Q8Cache(6, n_kv, bs, d, "e4m3")
    want.append(f64(k[:3]), f64(v[:3]), sl[:3])
    assert_cache(cache, want, [0, 1, 2])
    assert want.scales[1].max() == 0
    assert torch.equal(cache.records[3:], before[3:])
    assert torch.equal(cache.k_tail[:, :, 1:], torch.full_like(cache.k_tail[:, :, 1:], 5.0))


def build(lens, n_h, n_kv, d, bs, fmt, seed, outliers=False):
    """A cache with every sequence appended, the oracle's values of it, and queries."""
    rng = np.random.default_rng(seed)
    bt, blocks = tables(lens, bs, rng)
    g = torch.Generator().manual_seed(seed)
    n = int(sum(lens))
    k, v = (torch.randn(n, n_kv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    if outliers:
        k[..., 3] *= 20
        v *= torch.exp2(torch.randint(-12, 12, (n, 1, 1), generator=g)).to(torch.bfloat16)
    cache = pkv.alloc_q8_cache(blocks, n_kv, bs, d, len(lens), fmt, DEV)
    if n:
        sl = np.concatenate([slots_of(bt, s, 0, x, bs) for s, x in enumerate(lens)])
        ts = np.concatenate([np.full(x, s, np.int32) for s, x in enumerate(lens)])
        pkv.kv_quant_append_q8(k.to(DEV), v.to(DEV), dev(sl), dev(ts), cache)
    q = torch.randn(len(lens), n_h, d, generator=g).to(torch.bfloat16)
    sc = cache.scales.double().cpu().numpy()
    held = [f64(cache.k_codes.float()) * sc[:, :, 0, None, None], f64(cache.v_codes.float()) * sc[:, :, 1, None, None]]
    return cache, held, bt, q


def attend(q, cache, bt, ctx, scale, out_dtype=torch.float32, window=0, expect=0):
    err = err_flag()
    out = pkv.paged_decode_attn_q8(q.to(DEV), cache, dev(bt), dev(np.asarray(ctx, np.int32)), scale, window=window,
                                   out_dtype=out_dtype, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == expect, int(err.item())
    return out


def check_bf16(out, ref, v):
    """One rounding (2^-8 of the value at most) of a result within the fp32 bar and 2^-11 sum p |v| <=
    2^-11 max |v|: for a bf16 output and groups of over four heads p is rounded to fp16 once.  The rel-L2 bar of
    the bf16 cache's tests does not apply: it is the rounding of values with evenly spread mantissas
    (2^-8 / sqrt 3 over an octave, 1.7e-3), while a context of one token gives code * scale, whose few
    mantissas can all lie where the rounding costs up to 2^-8 = 3.9e-3."""
    got = f64(out)
    assert np.isfinite(got).all() and out.dtype == torch.bfloat16
    own = BAR_F32_MAXABS + 2.0 ** -11 * float(np.abs(v).max())
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + own * (1 + 2.0 ** -8)).all()


# The bars of the other attention tests hold here too: the codes are exact in fp16, q to 2^-39, p to
# 2^-22, sums and softmax in fp32; what differs from the bf16 kernel is smaller than its p (2^-16).
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 32), (64, 64), (128, 16), (128, 32), (128, 64)])
@pytest.mark.parametrize("n_h,n_kv", [(8, 8), (8, 2), (32, 8), (16, 1), (32, 1), (48, 1), (64, 1), (6, 3), (7, 1), (10, 2)])
def test_attention_sweep(fmt, d, bs, n_h, n_kv):
    lens = [0, 1, bs - 1, bs + 1, 3 * bs + 7, 2 * bs, 5 * bs, 70]
    cache, held, bt, q = build(lens, n_h, n_kv, d, bs, fmt, seed=n_h + bs)
    scale = 1 / math.sqrt(d)
    ref = oracle.paged_decode_attention(f64(q), *held, bt, lens, scale, bs)
    check_attention(attend(q, cache, bt, lens, scale), ref, "fp32")
    check_bf16(attend(q, cache, bt, lens, scale, torch.bfloat16), ref, held[1])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("bs,window", [(16, 1), (16, 15), (16, 40), (32, 33), (64, 100), (64, 7), (32, 1000)])
def test_attention_window(fmt, bs, window):
    lens = [1, 17, 64, 100, 255, 5 * bs]
    cache, held, bt, q = build(lens, 8, 2, 128, bs, fmt, seed=window)
    ref = oracle.paged_decode_attention(f64(q), *held, bt, lens, 0.1, bs, window=window)
    gone = bt.copy()
    for s, n in enumerate(lens):                               # released blocks before the window are not read
        gone[s, :max(0, n - window) // bs] = 10 ** 6
    check_attention(attend(q, cache, gone, lens, 0.1, window=window), ref, "window")


def test_attention_magnitudes():
    # queries from 2^-60 to 2^30, values over 24 octaves from block to block, keys with an outlier channel
    lens = [300, 33, 129, 64]
    cache, held, bt, q = build(lens, 8, 2, 64, 16, "e4m3", seed=2, outliers=True)
    q = (q.float() * torch.exp2(torch.tensor([-60.0, 0, 4, 30])).view(4, 1, 1)).to(torch.bfloat16)
    scale = [2.0 ** -3] * 3 + [2.0 ** -33]
    for s in range(4):
        ref = oracle.paged_decode_attention(f64(q[s:s + 1]), *held, bt[s:s + 1], lens[s:s + 1], scale[s], 16)
        out = f64(attend(q[s:s + 1], cache, bt[s:s + 1], lens[s:s + 1], scale[s]))
        # |error| <= (2 delta + 2^-19) sum_t p_t |v_t|: delta bounds the score's error, fp32 accumulation of d
        # products (d 2^-24 of sum |q k|) and a few roundings of the score itself
        k, v = (oracle.gather_sequence(held[i], bt[s], lens[s], 0, 16) for i in range(2))
        for h in range(4):
            qa = f64(q[s, h])
            delta = 2.0 ** -24 * 72 * scale[s] * (np.abs(k) @ np.abs(qa)).max()
            p = oracle.attention_weights(qa, k, scale[s])
            assert np.all(np.abs(out[0, h] - ref[0, h]) <= (2 * delta + 2.0 ** -19) * (p @ np.abs(v)) + 1e-30), (s, h)


def test_attention_rows_behind_the_context_do_not_count():
    # rows of the last block behind the context hold codes of NaN; their block's scale is finite
    lens = [5, 40, 17]
    cache, held, bt, q = build([n + 8 for n in lens], 8, 2, 64, 16, "e4m3", seed=6)
    for s, n in enumerate(lens):
        c = cache.records[int(bt[s, n // 16])]
        for kv in range(2):
            for r in range(n % 16, 16):
                for ch in range(64):
                    x, y, base = r % 16, ch % 32, kv * 16 * 64 + (ch // 32) * 512
                    if kv == 0:
                        b = (4 * (x % 8) + (y % 8) // 2) * 16 + 8 * (y // 16) + 4 * (x // 8) + 2 * ((y % 16) // 8) + y % 2
                    else:
                        b = (4 * (y % 8) + (x % 8) // 2) * 16 + 8 * (y // 16) + 4 * ((y % 16) // 8) + 2 * (x // 8) + x % 2
                    c[:, base + b] = 0x7f
    ref = oracle.paged_decode_attention(f64(q), *held, bt, lens, 0.125, 16)
    check_attention(attend(q, cache, bt, lens, 0.125), ref, "NaN codes behind the context")


def test_bad_blocks_and_lengths():
    lens = [100, 64, 30, 50]
    cache, held, bt, q = build(lens, 8, 2, 64, 16, "int8", seed=7)
    bad = bt.copy()
    bad[0, 2], bad[1, :], bad[2, 0] = held[0].shape[0], -5, 10 ** 9   # one inside, all, the first
    out = f64(attend(q, cache, bad, lens, 0.125, expect=pkv.DEV_BAD_BLOCK))
    assert np.array_equal(out[1], np.zeros_like(out[1]))
    for s, skip in ((0, [2]), (2, [0]), (3, [])):
        rows = [t for t in range(lens[s]) if t // 16 not in skip]
        for h in range(8):
            k, v = (np.stack([held[i][bt[s, t // 16], h // 4, t % 16] for t in rows]) for i in range(2))
            ref = oracle.attention_weights(f64(q[s, h]), k, 0.125) @ v
            assert np.abs(out[s, h] - ref).max() <= 5e-4
    over = np.array([100, 7 * 16 + 9, -4, 50], np.int32)       # clamped to the table and to zero
    out = f64(attend(q, cache, np.maximum(bt, 0), over, 0.125, expect=pkv.DEV_BAD_CTX))
    assert np.array_equal(out[2], np.zeros_like(out[2]))


@pytest.mark.parametrize("n_h,n_kv,lens", [(8, 2, [20000] + [3] * 300), (32, 1, [30000, 1, 0, 77]), (4, 4, [40001]),
                                           (8, 1, [9000] * 3 + [0] * 260)])
def test_long_and_many(n_h, n_kv, lens):
    # split segments (narrow and wide merge) and the plan kernel above 256 sequences
    cache, held, bt, q = build(lens, n_h, n_kv, 128, 32, "e4m3", seed=len(lens))
    scale = 1 / math.sqrt(128)
    ref = oracle.paged_decode_attention(f64(q), *held, bt, lens, scale, 32)
    a = attend(q, cache, bt, lens, scale)
    check_attention(a, ref, "long")
    assert torch.equal(a, attend(q, cache, bt, lens, scale))


# contexts around 64, 128 and 256 units (of 16 or 32 tokens) per segment, where the least length of a
# piece changes, and more sequences than one CTA plans for
@pytest.mark.parametrize("bs,unit", [(16, 16), (32, 32), (64, 32)])
@pytest.mark.parametrize("units", [63, 64, 127, 128, 255, 256])
def test_piece_lengths(bs, unit, units):
    lens = [units * unit, units * unit - unit + 1]
    cache, held, bt, q = build(lens, 4, 2, 64, bs, "e4m3", seed=units + bs)
    ref = oracle.paged_decode_attention(f64(q), *held, bt, lens, 0.125, bs)
    check_attention(attend(q, cache, bt, lens, 0.125), ref, "fp32")


def test_more_sequences_than_one_cta_plans():
    lens = [(7 * i) % 41 for i in range(300)]
    cache, held, bt, q = build(lens, 4, 2, 64, 16, "int8", seed=300)
    ref = oracle.paged_decode_attention(f64(q), *held, bt, lens, 0.125, 16)
    check_attention(attend(q, cache, bt, lens, 0.125), ref, "fp32")


def test_append_and_attend_in_a_graph_and_on_a_side_stream():
    lens = [33, 100, 5, 64]
    cache, _, bt, q = build(lens, 8, 2, 64, 16, "e4m3", seed=12)
    bt = np.concatenate([bt, np.full((4, 1), -1, np.int32)], 1)
    nxt = cache.records.shape[0] - 3                            # spare blocks
    for s, n in enumerate(lens):
        if n % 16 == 0:
            bt[s, n // 16] = nxt
            nxt += 1
    sl = dev(np.concatenate([slots_of(bt, s, n, n + 1, 16) for s, n in enumerate(lens)]))
    ts, ctx = torch.arange(4, dtype=torch.int32, device=DEV), dev(np.array(lens, np.int32) + 1)
    kn, vn = (torch.randn(4, 2, 64, device=DEV).to(torch.bfloat16) for _ in range(2))
    copies = [pkv.Q8CacheTensors(cache.records.clone(), cache.k_tail.clone(), cache.v_tail.clone(), "e4m3") for _ in range(3)]
    dq, dbt = q.to(DEV), dev(bt)
    ws = torch.empty(pkv.q8_workspace_bytes(4, 8, 2, 64, 16), dtype=torch.uint8, device=DEV)

    def step(c, out=None, stream=None):
        pkv.kv_quant_append_q8(kn, vn, sl, ts, c, stream=stream)
        return pkv.paged_decode_attn_q8(dq, c, dbt, ctx, 0.125, out=out, workspace=ws if stream is None else None, stream=stream)

    eager = step(copies[0])
    out = torch.empty_like(eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(copies[1], out)
    g.replay()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    side = step(copies[2], stream=st)                           # buffers of its own live as long as the stream's work
    torch.cuda.synchronize()
    assert torch.equal(eager, out) and torch.equal(eager, side)
    assert torch.equal(copies[0].records, copies[1].records) and torch.equal(copies[0].records, copies[2].records)


def test_refusals():
    c = pkv.alloc_q8_cache(4, 2, 16, 64, 2, "e4m3", DEV)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    sl, ts = torch.arange(2, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    q, bt, ctx = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 2, dtype=torch.int32, device=DEV), ts + 1
    bad_cache = pkv.Q8CacheTensors(c.records[:, :, :-16].contiguous(), c.k_tail, c.v_tail)
    for bad in (lambda: pkv.kv_quant_append_q8(k.half(), k, sl, ts, c), lambda: pkv.kv_quant_append_q8(k[:1], k, sl, ts, c),
                lambda: pkv.kv_quant_append_q8(k, k, sl.int(), ts, c), lambda: pkv.kv_quant_append_q8(k, k, sl, ts.long(), c),
                lambda: pkv.kv_quant_append_q8(k, k, sl, ts, bad_cache),
                lambda: pkv.paged_decode_attn_q8(q, bad_cache, bt, ctx, 1.0), lambda: pkv.paged_decode_attn_q8(q, c, bt, ctx, 1.0, window=-1),
                lambda: pkv.paged_decode_attn_q8(q[:, :7], c, bt, ctx, 1.0), lambda: pkv.paged_decode_attn_q8(q, c, bt[:1], ctx, 1.0),
                lambda: pkv.paged_decode_attn_q8(q, c, bt, ctx.long(), 1.0),
                lambda: pkv.paged_decode_attn_q8(q, c, bt, ctx, 1.0, out_dtype=torch.float16),
                lambda: pkv.paged_decode_attn_q8(q, c, bt, ctx, 1.0, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)),
                lambda: pkv.paged_decode_attn_q8(q, pkv.Q8CacheTensors(c.records, c.k_tail, c.v_tail, "e5m2"), bt, ctx, 1.0),
                lambda: pkv.q8_workspace_bytes(1, 65, 1, 64, 16)):
        with pytest.raises(pkv.PkvError):
            bad()
    out = pkv.paged_decode_attn_q8(q[:0], c, bt[:0], ctx[:0], 1.0)
    assert out.shape == (0, 8, 64)
    pkv.kv_quant_append_q8(k[:0], k[:0], sl[:0], ts[:0], c)
