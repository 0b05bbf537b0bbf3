"""Cases, plain forms and calls of the serving operators around the paged cache:

* ``rope``       rotary positions of a step's queries and keys, with the append of its K / V rows;
* ``q8_append``  quantize-on-append into the 8-bit cache (one scale per block of tokens and kv head);
* ``q8_attn``    decode attention over that cache;
* ``mass``       decode attention that adds each cached token's attention weight to its account;
* ``evict``      eviction down to a budget by those accounts.

``run`` computes them in elementary torch operations, or, where ``own`` is true, by the
framework's entry points.  ``exact`` is the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"


def listed():
    return [
        # one decode step of 64 sequences through a 32/8-head layer: a launch-bound call
        dict(name="rope_step64", op="rope", tokens=64, n_h=32, n_kv=8, d=128, bs=16, rot=128, inter=False,
             scaling="none", factor=1.0, far=4096),
        # a long prefill chunk of a model extended to eight times its trained length
        dict(name="rope_prefill16k", op="rope", tokens=16384, n_h=32, n_kv=8, d=128, bs=16, rot=128, inter=False,
             scaling="yarn", factor=8.0, far=131072),
        # an odd chunk with interleaved pairs over half of a small head
        dict(name="rope_partial_odd", op="rope", tokens=1013, n_h=25, n_kv=5, d=64, bs=32, rot=32, inter=True,
             scaling="linear", factor=4.0, far=16384),
        # one token of each of 64 sequences into unfinished blocks
        dict(name="q8_append_step64", op="q8_append", fmt="e4m3", seqs=64, new=1, n_kv=8, d=128, bs=16),
        # ragged prompts, continued from inside a block
        dict(name="q8_append_ragged", op="q8_append", fmt="int8", seqs=23, new=701, n_kv=8, d=128, bs=64),
        # the smallest serving batch: latency
        dict(name="q8_attn_small", op="q8_attn", fmt="e4m3", batch=4, lo=17, hi=255, n_h=8, n_kv=2, d=64, bs=16, window=0),
        # a 32/8-head layer, 64 sequences of 512 to 4096 tokens
        dict(name="q8_attn_b64", op="q8_attn", fmt="e4m3", batch=64, lo=512, hi=4096, n_h=32, n_kv=8, d=128, bs=16, window=0),
        # long contexts, large blocks
        dict(name="q8_attn_long", op="q8_attn", fmt="int8", batch=32, lo=8192, hi=32768, n_h=32, n_kv=8, d=128, bs=64, window=0),
        # the 32/8-head layer, with the accounts
        dict(name="mass_b64", op="mass", batch=64, lo=512, hi=4096, n_h=32, n_kv=8, d=128, bs=16),
        # one kv head for 32 query heads, a few long contexts of odd lengths
        dict(name="mass_mqa_long", op="mass", batch=8, lo=20011, hi=40009, n_h=32, n_kv=1, d=128, bs=32),
        # a serving batch cut to its budget
        dict(name="evict_b64", op="evict", batch=64, lo=2100, hi=4096, keep=2048, recent=256, n_kv=8, d=128, bs=16),
        # one long document cut to a quarter
        dict(name="evict_long", op="evict", batch=1, lo=131072, hi=131072, keep=32768, recent=1024, n_kv=8, d=128, bs=64),
    ]


def draw(rng):
    op = rng.choice(["rope", "q8_append", "q8_attn", "mass", "evict"])
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    d, bs, n_kv = rng.choice([64, 128]), rng.choice([16, 32, 64]), rng.choice([1, 2, 3, 4, 8, 32])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16, 32, 64])
    n_h = n_kv * (group if n_kv * group <= 64 else 1)
    fmt = rng.choice(["e4m3", "int8"])
    if op == "rope":
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d])
        t = log(1, max(1, 16384 * 48 * 128 // ((n_h + 2 * n_kv) * d) // 2))
        return dict(op=op, tokens=min(t, 30011), n_h=n_h, n_kv=n_kv, d=d, bs=bs, rot=rot, inter=rng.random() < 0.4,
                    scaling=rng.choice(["none", "linear", "ntk", "parts", "yarn"]), factor=rng.choice([2.0, 8.0, 32.0]),
                    far=log(1000, 1000000))
    if op == "q8_append":
        seqs = log(1, 256)
        new = 1 if rng.random() < 0.5 else log(2, max(2, min(8000, 16384 * 8 // (seqs * n_kv))))
        return dict(op=op, fmt=fmt, seqs=seqs, new=new, n_kv=n_kv, d=d, bs=bs)
    if op == "evict":
        b = log(1, 64)
        hi = log(40, max(48, min(131072, 64 * 4096 * 8 // (b * n_kv))))
        keep = max(1, int(hi * rng.uniform(0.1, 0.95)))
        return dict(op=op, batch=b, lo=max(1, hi // 2), hi=hi, keep=keep, recent=rng.randrange(0, keep), n_kv=n_kv, d=d, bs=bs)
    b = log(1, 200)
    hi = log(1, max(2, min(131072, 32 * 20000 * 8 // (b * n_kv), 400000000 // (b * n_h))))
    c = dict(op=op, batch=b, lo=max(1, hi // 8), hi=hi, n_h=n_h, n_kv=n_kv, d=d, bs=bs)
    if op == "q8_attn":
        c.update(fmt=fmt, window=log(1, hi) if rng.random() < 0.25 else 0)
    return c


# ---- sizes that a case fixes (the seed draws the values) ------------------------------------------
def lengths(n, lo, hi):
    """n lengths spread over [lo, hi], both ends among them."""
    u = (np.arange(n) * 0.6180339887498949) % 1.0
    return np.rint(lo + (hi - lo) * (u / max(u.max(), 1e-9) if n > 1 else np.ones(1))).astype(np.int32)


def append_sizes(c):
    """(new tokens, rows of the open block already there) of each sequence."""
    n = lengths(c["seqs"], max(1, c["new"] // 3), c["new"]) if c["new"] > 1 else np.ones(c["seqs"], np.int32)
    return n, ((np.arange(c["seqs"]) * 7 + 3) % c["bs"]).astype(np.int32)


def work(c):
    if c["op"] == "rope":
        e = c["tokens"] * (c["n_h"] + 2 * c["n_kv"]) * c["d"]
        return {"bytes": 4 * e + 12 * c["tokens"], "flops": 3 * c["tokens"] * (c["n_h"] + c["n_kv"]) * c["rot"]}
    if c["op"] == "q8_append":
        n, r0 = (x.astype(np.int64) for x in append_sizes(c))
        end = r0 + n
        rows = int(end.sum())                                  # rows quantized: old ones of the open blocks and new ones
        tails = int(np.where(end % c["bs"] > 0, np.minimum(n, end % c["bs"]), 0).sum())
        per = 2 * c["n_kv"] * c["d"]                           # K and V channels of a row
        return {"bytes": per * (2 * rows + rows + 2 * tails) + 12 * int(n.sum()), "flops": 3 * per * rows}
    ctx = lengths(c["batch"], c["lo"], c["hi"]).astype(np.int64)
    if c["op"] == "evict":
        K = np.minimum(ctx, c["keep"])
        rec = np.minimum(c["recent"], K)
        free = np.maximum(ctx - rec, 1)
        moves = np.where(ctx > K, np.minimum(rec, ctx - K) + np.maximum(ctx - K - rec, 0) * (K - rec) / free, 0).sum()
        return {"bytes": float(c["n_kv"] * (8 * ctx.sum() + 4 * K.sum() + moves * 8 * c["d"])), "flops": float(c["n_kv"] * ctx.sum())}
    seen = np.minimum(ctx, c["window"]) if c.get("window") else ctx
    t, io = int(seen.sum()), 4 * c["batch"] * c["n_h"] * c["d"]
    per_token = 2 * c["d"] * (1 if c["op"] == "q8_attn" else 2) + (8 if c["op"] == "mass" else 0)
    return {"bytes": t * c["n_kv"] * per_token + io, "flops": 4 * t * c["n_h"] * c["d"]}


# ---- inputs -----------------------------------------------------------------------------------------
def gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7fffffff)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def tables(c, lens, seed):
    """Physical blocks of each sequence, drawn from a shuffled pool a fifth larger than needed."""
    bs = c["bs"]
    nb = -(-np.asarray(lens, np.int64) // bs)
    blocks = int(nb.sum()) + max(1, int(nb.sum()) // 5)
    perm = np.random.RandomState(seed & 0x7fffffff).permutation(blocks).astype(np.int32)
    bt = np.full((len(nb), max(1, int(nb.max()))), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(nb)])
    for s in range(len(nb)):
        bt[s, :nb[s]] = perm[at[s]:at[s + 1]]
    return bt, blocks


def rope_freqs(c):
    """Inverse wavelengths of the channel pairs after the scaling, and the amplitude."""
    r, base, f, length = c["rot"], 10000.0, c["factor"], max(64.0, c["far"] / c["factor"])
    j = np.arange(r // 2, dtype=np.float64)
    if c["scaling"] == "ntk":
        base = base * f ** (r / (r - 2.0))
    inv = base ** (-2.0 * j / r)
    if c["scaling"] == "linear":
        inv = inv / f
    if c["scaling"] == "parts":                                 # by the turns that a pair makes over the trained length
        w = np.clip((length * inv / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0, 1)
        inv = w * inv + (1 - w) * inv / f
    if c["scaling"] == "yarn":                                  # by the pair's place between those of 32 turns and of one
        place = lambda turns: r * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), r - 1)
        w = 1 - np.clip((j - lo) / max(hi - lo, 0.001), 0, 1)
        return w * inv + (1 - w) * inv / f, 0.1 * math.log(f) + 1.0
    return inv, 1.0


def prepare(c, seed):
    g, s = gen(seed), dict(c)
    op, d, bs, n_kv = c["op"], c["d"], c["bs"], c["n_kv"]
    if op == "rope":
        n, n_h = c["tokens"], c["n_h"]
        qkv = normal(g, n, (n_h + 2 * n_kv) * d)                # as the fused projection leaves it
        q, k, v = qkv.split([n_h * d, n_kv * d, n_kv * d], 1)
        s.update(q=q.view(n, n_h, d), k=k.view(n, n_kv, d), v=v.view(n, n_kv, d))
        s["positions"] = torch.randint(0, c["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
        blocks = -(-n // bs) + 2
        s["slots"] = torch.randperm(blocks * bs, generator=g, device=DEV)[:n]
        s["k_pool"], s["v_pool"] = normal(g, blocks, n_kv, bs, d), normal(g, blocks, n_kv, bs, d)
        s["q_out"] = torch.empty(n, n_h, d, dtype=torch.bfloat16, device=DEV)
        inv, s["amp"] = rope_freqs(c)
        s["inv"] = torch.as_tensor(inv, device=DEV)
        return s
    if op == "q8_append":
        n, r0 = append_sizes(c)
        bt, blocks = tables(c, r0 + n, seed)
        seq = np.repeat(np.arange(len(n)), n)
        row = np.concatenate([a + np.arange(b) for a, b in zip(r0, n)])
        s["slots"] = torch.as_tensor(bt[seq, row // bs].astype(np.int64) * bs + row % bs, device=DEV)
        s["tail_seq"] = torch.as_tensor(seq.astype(np.int32), device=DEV)
        s["k"], s["v"] = normal(g, len(seq), n_kv, d), normal(g, len(seq), n_kv, d)
        s["k_tail"], s["v_tail"] = normal(g, c["seqs"], n_kv, bs, d), normal(g, c["seqs"], n_kv, bs, d)
        s["records"] = torch.zeros(blocks, n_kv, 2 * bs * d + 16, dtype=torch.uint8, device=DEV)
        return s
    ctx = lengths(c["batch"], c["lo"], c["hi"])
    bt, blocks = tables(c, ctx, seed)
    s["bt"], s["ctx"] = torch.as_tensor(bt, device=DEV), torch.as_tensor(ctx, device=DEV)
    T = bt.shape[1] * bs
    if op == "q8_attn":
        s["q"], s["out"] = normal(g, c["batch"], c["n_h"], d), torch.empty(c["batch"], c["n_h"], d, dtype=torch.bfloat16, device=DEV)
        rec = torch.zeros(blocks, n_kv, 2 * bs * d + 16, dtype=torch.uint8, device=DEV)
        x = torch.randn(blocks, n_kv, 2, bs * d, generator=g, device=DEV) * (0.5 + torch.rand(blocks, n_kv, 2, 1, generator=g, device=DEV))
        codes, scale = quantize(x, c["fmt"])
        rec[:, :, :2 * bs * d] = codes.view(blocks, n_kv, -1)
        rec[:, :, 2 * bs * d:2 * bs * d + 8].view(torch.float32)[:] = scale.view(blocks, n_kv, 2)
        s["records"] = rec
        s["k_tail"], s["v_tail"] = (torch.zeros(c["batch"], n_kv, bs, d, dtype=torch.bfloat16, device=DEV) for _ in "kv")
        return s
    s["k_pool"], s["v_pool"] = normal(g, blocks, n_kv, bs, d), normal(g, blocks, n_kv, bs, d)
    if op == "mass":
        s["q"], s["out"] = normal(g, c["batch"], c["n_h"], d), torch.empty(c["batch"], c["n_h"], d, dtype=torch.bfloat16, device=DEV)
        s["mass"] = torch.rand(c["batch"], n_kv, T, generator=g, device=DEV) * (torch.arange(T, device=DEV) < s["ctx"][:, None, None])
        return s
    e = torch.rand(c["batch"], n_kv, T, generator=g, device=DEV)
    s["mass"] = -torch.log(1 - e) * (torch.arange(T, device=DEV) < s["ctx"][:, None, None])
    # the rows an earlier eviction left, in its order; what came after is in order
    s["kept"] = torch.minimum(s["ctx"], torch.full_like(s["ctx"], max(1, c["keep"] // 2)))
    s["dropped"] = torch.full_like(s["ctx"], 5)
    p = torch.rand(c["batch"], n_kv, T, generator=g, device=DEV) + 2.0 * (torch.arange(T, device=DEV) >= s["kept"][:, None, None])
    s["positions"] = torch.argsort(torch.argsort(p, dim=-1), dim=-1).to(torch.int32) + 2
    s["keep"] = torch.full_like(s["ctx"], c["keep"])
    s["o_mass"], s["o_positions"] = torch.zeros_like(s["mass"]), torch.zeros_like(s["positions"])
    s["o_kept"], s["o_dropped"], s["new_lens"] = (torch.zeros_like(s["ctx"]) for _ in range(3))
    return s


# ---- plain forms ------------------------------------------------------------------------------------
def rotate_plain(x, cos, sin, rot, inter):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1 if inter else -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


def rope_plain(s):
    ang = s["positions"].double()[:, None] * s["inv"]
    cos, sin = (torch.cos(ang) * s["amp"]).float()[:, None], (torch.sin(ang) * s["amp"]).float()[:, None]
    s["q_out"].copy_(rotate_plain(s["q"], cos, sin, s["rot"], s["inter"]))
    blk, row = s["slots"] // s["bs"], s["slots"] % s["bs"]
    s["k_pool"][blk, :, row] = rotate_plain(s["k"], cos, sin, s["rot"], s["inter"])
    s["v_pool"][blk, :, row] = s["v"]


def quantize(x, fmt):
    """Codes (as bytes) and scale of groups along the last axis."""
    most = 448.0 if fmt == "e4m3" else 127.0
    big = x.abs().amax(-1, keepdim=True)
    some = big >= 2.0 ** -110
    scale = torch.where(some, big / most, 0.0)
    y = x * torch.where(some, most / big, 0.0)
    if fmt == "e4m3":
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale[..., 0]
    return y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8), scale[..., 0]


def tiles(x, keys):
    """[.., bs, d] values in the record's order: 16-token tiles of 32 channels, by lane (gid, tig), 16 bytes a lane."""
    *n, bs, d = x.shape
    z = len(n)
    if keys:    # token = 16 tt + 8 hi + gid, channel = 32 j + 16 ks + 8 half + 2 tig + b
        y = x.reshape(*n, bs // 16, 2, 8, d // 32, 2, 2, 4, 2)
        order = [0, 3, 2, 6, 4, 1, 5, 7]
    else:       # token = 16 tt + 8 half + 2 tig + b, channel = 32 j + 16 md + 8 hi + gid
        y = x.reshape(*n, bs // 16, 2, 4, 2, d // 32, 2, 2, 8)
        order = [0, 4, 7, 2, 5, 6, 1, 3]
    return y.permute(*range(z), *[z + i for i in order]).reshape(*n, bs * d)


def untiles(x, bs, d, keys):
    *n, _ = x.shape
    z = len(n)
    y = x.reshape(*n, bs // 16, d // 32, 8, 4, 2, 2, 2, 2)
    order = [0, 5, 2, 1, 4, 6, 3, 7] if keys else [0, 6, 3, 7, 1, 4, 5, 2]
    return y.permute(*range(z), *[z + i for i in order]).reshape(*n, bs, d)


def q8_append_plain(s):
    bs, d, slots, seq = s["bs"], s["d"], s["slots"], s["tail_seq"].long()
    n = slots.numel()
    blk, row = slots // bs, slots % bs
    at = torch.arange(n, device=DEV)
    first = torch.cat([torch.ones(1, dtype=torch.bool, device=DEV), blk[1:] != blk[:-1]]).nonzero()[:, 0]   # first new row of each block
    many = torch.diff(first, append=torch.tensor([n], device=DEV))
    r = torch.arange(bs, device=DEV)
    r0, end = row[first][:, None], (row[first] + many)[:, None]
    new, old = (r >= r0) & (r < end), r < r0
    src = (first[:, None] + r - r0).clamp(0, n - 1)
    out = {}
    for name, x, tail in (("k", s["k"], s["k_tail"]), ("v", s["v"], s["v_tail"])):
        rows = torch.where(new[:, :, None, None], x[src], tail[seq[first]].transpose(1, 2)).float()
        rows = torch.where((new | old)[:, :, None, None], rows, 0.0).transpose(1, 2)                        # [block][kv head][row][channel]
        codes, scale = quantize(rows.flatten(-2), s["fmt"])
        out[name] = tiles(codes.view(*rows.shape), name == "k"), scale
    rec, b = s["records"], blk[first]
    rec[b] = torch.cat([out["k"][0], out["v"][0], torch.zeros(len(b), s["n_kv"], 16, dtype=torch.uint8, device=DEV)], -1)
    rec[b, :, 2 * bs * d:2 * bs * d + 8] = torch.stack([out["k"][1], out["v"][1]], -1).view(torch.uint8)
    last = torch.cat([seq[1:] != seq[:-1], torch.ones(1, dtype=torch.bool, device=DEV)])
    lens = row[last.nonzero()[:, 0]] + 1                        # rows of each sequence's last block
    ends = torch.zeros(s["k_tail"].shape[0], dtype=torch.long, device=DEV).index_put_((seq[last],), at[last])
    rows_of = torch.zeros_like(ends).index_put_((seq[last],), lens)
    t = ((blk == blk[ends[seq]]) & (rows_of[seq] < bs)).nonzero()[:, 0]                                     # new rows of open blocks
    s["k_tail"][seq[t], :, row[t]] = s["k"][t]
    s["v_tail"][seq[t], :, row[t]] = s["v"][t]


def codes_of(s):
    bs, d, rec = s["bs"], s["d"], s["records"]
    kind = torch.float8_e4m3fn if s["fmt"] == "e4m3" else torch.int8
    return rec[:, :, :2 * bs * d].view(kind), rec[:, :, 2 * bs * d:2 * bs * d + 8].view(torch.float32)


def logits_plain(q, k, scale):
    """[B][n_h][d] x [B][n_kv][T][d] -> [B][n_kv][G][T]"""
    B, n_h, d = q.shape
    return torch.matmul(q.float().view(B, k.shape[1], -1, d), k.transpose(-1, -2)) * scale


def attend_plain(x, v, ctx, window=0):
    t = torch.arange(x.shape[-1], device=DEV)
    seen = (t < ctx[:, None]) & ((t >= ctx[:, None] - window) | (window == 0))
    x = torch.where(seen[:, None, None], x, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    return torch.matmul(p, v).flatten(1, 2), p


def q8_attn_plain(s):
    bs, d = s["bs"], s["d"]
    codes, scale = codes_of(s)
    bt = s["bt"].long().clamp(min=0)
    codes, scale = codes.view(torch.uint8)[bt].view(codes.dtype), scale[bt]                                 # [B][blocks][kv head][...]
    kv = [(untiles(codes[..., i * bs * d:(i + 1) * bs * d].view(torch.uint8), bs, d, i == 0).view(codes.dtype).float()
           * scale[..., i, None, None]).transpose(1, 2).flatten(2, 3) for i in range(2)]
    o, _ = attend_plain(logits_plain(s["q"], kv[0], d ** -0.5), kv[1], s["ctx"], s["window"])
    s["out"].copy_(o)


def gathered(pool, bt):
    return pool[bt.long().clamp(min=0)].transpose(1, 2).flatten(2, 3).float()


def mass_plain(s):
    k, v = gathered(s["k_pool"], s["bt"]), gathered(s["v_pool"], s["bt"])
    o, p = attend_plain(logits_plain(s["q"], k, s["d"] ** -0.5), v, s["ctx"])
    s["out"].copy_(o)
    s["mass"] += p.sum(2)


def evict_plain(s):
    n, bs = s["ctx"][:, None, None], s["bs"]
    keep = torch.minimum(s["keep"], s["ctx"])[:, None, None]
    cut = n > keep
    r = torch.arange(s["mass"].shape[-1], device=DEV)
    kept, dropped = s["kept"][:, None, None], s["dropped"][:, None, None]
    pos = torch.where(r < kept, s["positions"], dropped + r)
    recent = pos >= dropped + n - keep.clamp(max=s["recent"])
    key = torch.where(r < n, torch.where(recent, math.inf, s["mass"]), -math.inf)
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices
    stays = torch.zeros_like(key, dtype=torch.bool).scatter_(-1, best, (r < keep).expand_as(best))
    hb, hg, hole = (~stays & (r < keep)).nonzero(as_tuple=True)             # the i-th hole takes the i-th kept row behind the budget
    mb, mg, move = (stays & (r >= keep)).nonzero(as_tuple=True)
    bt = s["bt"].long()
    for pool in (s["k_pool"], s["v_pool"]):
        pool[bt[hb, hole // bs], hg, hole % bs] = pool[bt[mb, move // bs], mg, move % bs]
    mass = torch.where(r < keep, s["mass"], 0.0)
    mass[hb, hg, hole] = s["mass"][mb, mg, move]
    newpos = pos.clone()
    newpos[hb, hg, hole] = pos[mb, mg, move]
    s["o_mass"].copy_(torch.where(r < n, mass, s["o_mass"]))
    s["o_positions"].copy_(torch.where(torch.where(cut, r < keep, r < kept), newpos, s["o_positions"]))
    s["new_lens"].copy_(keep[:, 0, 0])
    s["o_kept"].copy_(torch.where(cut, keep, kept)[:, 0, 0])
    s["o_dropped"].copy_((dropped + n - keep)[:, 0, 0])


# ---- one pass ---------------------------------------------------------------------------------------
def run_own(s):
    import paged_kv_cache_175_gb300 as pkv
    op = s["op"]
    if op == "rope":
        table = pkv.rope_table(s["d"], s["rot"], interleaved=s["inter"], scaling=s["scaling"], factor=s["factor"],
                               original_len=max(64.0, s["far"] / s["factor"]), **(dict(low=1.0, high=4.0) if s["scaling"] == "parts" else {}))
        pkv.rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], table, s["k_pool"], s["v_pool"], q_out=s["q_out"])
    elif op == "q8_append":
        cache = pkv.Q8CacheTensors(s["records"], s["k_tail"], s["v_tail"], s["fmt"])
        pkv.kv_quant_append_q8(s["k"], s["v"], s["slots"], s["tail_seq"], cache)
    elif op == "q8_attn":
        cache = pkv.Q8CacheTensors(s["records"], s["k_tail"], s["v_tail"], s["fmt"])
        if "workspace" not in s:
            s["workspace"] = torch.empty(pkv.q8_workspace_bytes(s["batch"], s["n_h"], s["n_kv"], s["d"], s["bs"], s["fmt"]),
                                         dtype=torch.uint8, device=DEV)
        pkv.paged_decode_attn_q8(s["q"], cache, s["bt"], s["ctx"], s["d"] ** -0.5, window=s["window"], out=s["out"],
                                 workspace=s["workspace"])
    elif op == "mass":
        if "workspace" not in s:
            s["workspace"] = torch.empty(pkv.mass_workspace_bytes(s["batch"], s["n_h"], s["n_kv"], s["d"], s["bs"], s["bt"].shape[1]),
                                         dtype=torch.uint8, device=DEV)
        pkv.paged_decode_attn_mass(s["q"], s["k_pool"], s["v_pool"], s["bt"], s["ctx"], s["d"] ** -0.5, s["mass"],
                                   out=s["out"], workspace=s["workspace"])
    else:
        if "workspace" not in s:
            s["workspace"] = torch.empty(pkv.evict_workspace_bytes(s["batch"], s["n_kv"], s["bs"], s["bt"].shape[1]),
                                         dtype=torch.uint8, device=DEV)
        pkv.kv_evict(s["k_pool"], s["v_pool"], s["bt"], s["ctx"], s["keep"], s["recent"],
                     pkv.EvictState(s["mass"], s["positions"], s["kept"], s["dropped"]),
                     out=pkv.EvictState(s["o_mass"], s["o_positions"], s["o_kept"], s["o_dropped"]),
                     new_lens=s["new_lens"], workspace=s["workspace"])


PLAIN = {"rope": rope_plain, "q8_append": q8_append_plain, "q8_attn": q8_attn_plain, "mass": mass_plain, "evict": evict_plain}


def run(s):
    if own:
        run_own(s)
    else:
        PLAIN[s["op"]](s)
    if s["op"] == "rope":
        return s["q_out"], s["k_pool"], s["v_pool"]
    if s["op"] == "q8_append":
        return (*codes_of(s), s["k_tail"], s["v_tail"])
    if s["op"] == "q8_attn":
        return s["out"]
    if s["op"] == "mass":
        return s["out"], s["mass"]
    return s["k_pool"], s["v_pool"], s["o_mass"], s["o_positions"], s["o_kept"], s["o_dropped"], s["new_lens"]


# ---- the definitions in 64 bits ---------------------------------------------------------------------
def exact_attention(q, k, v, scale):
    """Softmax attention of heads q [n_h][d] over k, v [n_kv][T][d]: outputs and weights."""
    G = q.shape[0] // k.shape[0]
    o, w = [], []
    for g in range(k.shape[0]):
        x = q[g * G:(g + 1) * G].double() @ k[g].double().T * scale
        p = torch.softmax(x, -1)
        o.append(p @ v[g].double())
        w.append(p.sum(0))
    return torch.cat(o), torch.stack(w)


def lane_bytes(bs, d, keys):
    """Byte of element (token, channel) inside its part of a record."""
    t, ch = np.meshgrid(np.arange(bs), np.arange(d), indexing="ij")
    if not keys:    # values: tokens along a lane's bytes, channels over the lanes
        line, col = ch % 16, t % 16
        group, step = ch // 32, (ch // 16) % 2
    else:
        line, col = t % 16, ch % 16
        group, step = ch // 32, (ch // 16) % 2
    lane = (line % 8) * 4 + (col % 8) // 2
    return (t // 16) * 16 * d + group * 512 + lane * 16 + step * 8 + (line // 8) * 4 + (col // 8) * 2 + col % 2


def exact(c, seed):
    s = prepare(c, seed)
    bs, d = c["bs"], c["d"]
    if c["op"] == "rope":
        z = torch.polar(torch.full((), float(s["amp"]), dtype=torch.float64, device=DEV), s["positions"].double()[:, None] * s["inv"])[:, None]
        res = []
        for x in (s["q"].double(), s["k"].double()):
            y, r = x.clone(), c["rot"]
            i = torch.arange(0, r, 2, device=DEV) if c["inter"] else torch.arange(r // 2, device=DEV)
            j = i + (1 if c["inter"] else r // 2)
            w = torch.complex(x[..., i], x[..., j]) * z
            y[..., i], y[..., j] = w.real, w.imag
            res.append(y)
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        b, row = torch.div(s["slots"], bs, rounding_mode="floor"), torch.remainder(s["slots"], bs)
        kp[b, :, row], vp[b, :, row] = res[1], s["v"].double()
        return res[0], kp, vp
    if c["op"] == "q8_append":
        if c["fmt"] == "int8" and len(s["slots"]) > 100000:
            return None
        codes = torch.zeros(s["records"].shape[0], c["n_kv"], 2 * bs * d, dtype=torch.float64, device=DEV)
        scales = torch.zeros(s["records"].shape[0], c["n_kv"], 2, dtype=torch.float64, device=DEV)
        n, r0 = append_sizes(c)
        slots, at = s["slots"].cpu().numpy(), 0
        tails = [s["k_tail"].double(), s["v_tail"].double()]
        place = [torch.as_tensor(lane_bytes(bs, d, i == 0), device=DEV).flatten() for i in range(2)]
        for q in range(c["seqs"]):
            end, done = int(r0[q] + n[q]), int(r0[q])
            before = [t[q].clone() for t in tails]
            while done < end:
                upto = min(end, done // bs * bs + bs)
                phys, lo, m = int(slots[at]) // bs, done % bs, upto - done
                for i, x in enumerate((s["k"], s["v"])):
                    rows = torch.zeros(c["n_kv"], bs, d, dtype=torch.float64, device=DEV)
                    rows[:, :lo] = before[i][:, :lo]
                    rows[:, lo:lo + m] = x[at:at + m].double().transpose(0, 1)
                    big = rows.abs().amax((1, 2), keepdim=True)
                    y = rows / big
                    if c["fmt"] == "e4m3":     # nearest of the 8-bit floats: step 2^(e-3), 2^-9 below 2^-6
                        y = y * 448.0
                        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                        y = torch.round(y / step) * step
                    else:
                        y = torch.round(y * 127.0)
                    codes[phys, :, i * bs * d + place[i]] = y.flatten(1)
                    scales[phys, :, i] = (big / (448.0 if c["fmt"] == "e4m3" else 127.0))[:, 0, 0]
                    if upto == end and end % bs:
                        tails[i][q][:, lo:lo + m] = x[at:at + m].double().transpose(0, 1)
                at, done = at + m, upto
        return (codes if c["fmt"] == "e4m3" else None), scales, tails[0], tails[1]
    ctx = lengths(c["batch"], c["lo"], c["hi"])
    bt = s["bt"].long()
    if c["op"] == "q8_attn":
        kind = torch.float8_e4m3fn if c["fmt"] == "e4m3" else torch.int8
        place = [torch.as_tensor(lane_bytes(bs, d, i == 0), device=DEV).flatten() for i in range(2)]
        out = []
        for b in range(c["batch"]):
            n = int(ctx[b])
            rec = s["records"][bt[b, :-(-n // bs)]]
            scale = rec[..., 2 * bs * d:2 * bs * d + 8].contiguous().view(torch.float32).double()
            kv = []
            for i in range(2):
                x = rec[..., i * bs * d + place[i]].view(kind).double() * scale[..., i, None]
                x = x.view(-1, c["n_kv"], bs, d).transpose(0, 1).flatten(1, 2)[:, :n]
                kv.append(x[:, max(0, n - c["window"]):] if c["window"] else x)
            out.append(exact_attention(s["q"][b], kv[0], kv[1], d ** -0.5)[0])
        return torch.stack(out)
    if c["op"] == "mass":
        out, mass = [], s["mass"].double()
        for b in range(c["batch"]):
            n = int(ctx[b])
            k, v = (p[bt[b, :-(-n // bs)]].transpose(0, 1).flatten(1, 2)[:, :n] for p in (s["k_pool"], s["v_pool"]))
            o, w = exact_attention(s["q"][b], k, v, d ** -0.5)
            out.append(o)
            mass[b, :, :n] += w
        return torch.stack(out), mass
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    mass, kept = s["mass"].cpu().numpy().astype(np.float64), s["kept"].cpu().numpy()
    posn, table, drop = s["positions"].cpu().numpy(), s["bt"].cpu().numpy(), s["dropped"].cpu().numpy()
    o = s["o_mass"].cpu().numpy().astype(np.float64)
    src, dst = [], []
    for b in range(c["batch"]):
        n, K = int(ctx[b]), min(int(ctx[b]), c["keep"])
        for g in range(c["n_kv"]):
            p = np.arange(n) + drop[b]
            p[:min(n, kept[b])] = posn[b, g, :min(n, kept[b])]
            forced = p >= drop[b] + n - min(c["recent"], K)
            order = np.lexsort((np.arange(n), -mass[b, g, :n], ~forced))[:K]
            stay = np.zeros(n, bool)
            stay[order] = True
            holes, moves = np.flatnonzero(~stay[:K]), K + np.flatnonzero(stay[K:])
            row = np.where(np.arange(n) < K, mass[b, g, :n], 0.0)
            row[holes] = mass[b, g, moves]
            o[b, g, :n] = row
            slot = lambda r: (table[b, r // bs].astype(np.int64) * c["n_kv"] + g) * bs + r % bs  # noqa: E731,B023
            src.append(slot(moves))
            dst.append(slot(holes))
    src, dst = (torch.as_tensor(np.concatenate(x), device=DEV) for x in (src, dst))
    for p in (kp, vp):
        p.view(-1, d)[dst] = p.view(-1, d)[src]
    return kp, vp, torch.as_tensor(o, device=DEV), None, None, None, None
