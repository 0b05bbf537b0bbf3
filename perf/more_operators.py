"""Cases, plain forms and calls of the operators for drafted tokens and for the latent cache:

* ``tree``     attention for a tree of drafted tokens over the paged bf16 cache;
* ``accept``   the accepted path's rows moved to the front of the drafted ones, in all layers' pools;
* ``lappend``  norm of the latent vectors, rotation of the shared key part and of the queries' part, append
               to the paged latent cache;
* ``latent``   attention over that cache (absorbed form), of one token or a tree of them per sequence.

``run`` computes them in elementary torch operations, or, where ``own`` is true, by the framework's
entry points.  ``exact`` is the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"


def listed():
    return [
        # one interactive sequence, a small tree: latency
        dict(name="tree_one", op="tree", batch=1, drafts=8, lo=333, hi=333, n_h=32, n_kv=8, d=128, bs=16, mask=True, f32=False),
        # a serving batch of the 32/8-head layer, trees of up to 16 tokens
        dict(name="tree_b64", op="tree", batch=64, drafts=16, lo=512, hi=4096, n_h=32, n_kv=8, d=128, bs=16, mask=True, f32=False),
        # long documents with wide trees, 64/8 heads: 512 query rows for every cached one
        dict(name="tree_long", op="tree", batch=8, drafts=64, lo=8192, hi=32768, n_h=64, n_kv=8, d=128, bs=64, mask=True, f32=False),
        # ragged chains (the last tokens of a prompt, or a draft without branches), small odd heads, 32-bit output
        dict(name="tree_chain_odd", op="tree", batch=23, drafts=9, lo=17, hi=2049, n_h=25, n_kv=5, d=64, bs=32, mask=False, f32=True),
        # one sequence through a few heads of a latent cache: latency
        dict(name="latent_one", op="latent", batch=1, drafts=1, lo=301, hi=301, n_h=16, latent=512, rope=64, bs=64, mask=False, f32=False),
        # a decode step of 64 sequences with the heads of one of several devices
        dict(name="latent_b64", op="latent", batch=64, drafts=1, lo=512, hi=4096, n_h=16, latent=512, rope=64, bs=64, mask=False, f32=False),
        # all 128 heads over long contexts: near the border between memory and tensor cores
        dict(name="latent_h128", op="latent", batch=32, drafts=1, lo=2048, hi=16384, n_h=128, latent=512, rope=64, bs=64, mask=False, f32=False),
        # trees of drafted tokens over the latent cache, small blocks, odd lengths
        dict(name="latent_tree", op="latent", batch=12, drafts=8, lo=1021, hi=8191, n_h=32, latent=512, rope=64, bs=16, mask=True, f32=False),
        # one decode step into the latent cache
        dict(name="lappend_step64", op="lappend", tokens=64, n_h=128, latent=512, rope=64, bs=64, norm=True, inter=True, far=16384),
        # a long prompt chunk into it
        dict(name="lappend_prompt", op="lappend", tokens=16001, n_h=16, latent=512, rope=64, bs=64, norm=True, inter=False, far=131072),
        # accepted paths of 64 sequences, eight layers of keys and values
        dict(name="accept_b64", op="accept", batch=64, drafts=16, lo=128, hi=512, n_kv=8, width=128, pools=16, bs=16),
        # a few wide trees over the latent caches of many layers
        dict(name="accept_latent", op="accept", batch=4, drafts=64, lo=500, hi=2000, n_kv=1, width=576, pools=40, bs=64),
    ]


def draw(rng):
    op = rng.choice(["tree", "tree", "accept", "lappend", "latent", "latent"])
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))  # noqa: E731
    bs = rng.choice([16, 32, 64])
    if op == "tree":
        d, n_kv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8, 16])
        group = rng.choice([1, 2, 4, 5, 7, 8, 16, 32, 64])
        n_h = n_kv * (group if n_kv * group <= 64 else 1)
        drafts = log(1, 64)
        b = log(1, 128)
        hi = log(1, min(131072, 160000 * 8 // (b * n_kv) + 1, 300000000 // (b * drafts * n_h) + 1))
        return dict(op=op, batch=b, drafts=drafts, lo=max(0, hi // 8), hi=hi, n_h=n_h, n_kv=n_kv, d=d, bs=bs,
                    mask=rng.random() < 0.7, f32=rng.random() < 0.3)
    if op == "latent":
        n_h = rng.choice([1, 8, 12, 16, 20, 32, 40, 64, 128])
        drafts = 1 if rng.random() < 0.5 else log(2, 32)
        b = log(1, min(128, 32768 // (drafts * n_h)))
        hi = log(1, min(131072, 290000 // b + 1, 36000000 // (b * drafts * n_h) + 1))
        latent, rope = rng.choice([(512, 64), (512, 64), (256, 64), (256, 32), (512, 32)])
        return dict(op=op, batch=b, drafts=drafts, lo=max(0, hi // 8), hi=hi, n_h=n_h, latent=latent, rope=rope, bs=bs,
                    mask=rng.random() < 0.7, f32=rng.random() < 0.3)
    if op == "lappend":
        n_h = rng.choice([1, 8, 12, 16, 20, 32, 40, 64, 128])
        latent, rope = rng.choice([(512, 64), (256, 64), (256, 32), (512, 32)])
        return dict(op=op, tokens=log(1, 16001 * 1600 // (576 + n_h * 64)), n_h=n_h, latent=latent, rope=rope, bs=bs,
                    norm=rng.random() < 0.8, inter=rng.random() < 0.5, far=log(1000, 1000000))
    n_kv, width = rng.choice([(1, 576), (1, 320), (8, 128), (4, 64), (1, 128), (5, 64)])
    pools, drafts = rng.choice([1, 2, 8, 16, 40]), log(1, 64)
    b = log(1, max(1, min(128, 16000000 // (pools * n_kv * width * drafts))))
    hi = log(1, max(1, 320000000 // (b * n_kv * width * pools * 4)))
    return dict(op=op, batch=b, drafts=drafts, lo=max(0, hi // 4), hi=hi, n_kv=n_kv, width=width, pools=pools, bs=bs)


# ---- sizes that a case fixes (the seed draws the values) ------------------------------------------
def spread(n, lo, hi, at=0.0):
    """n whole numbers spread over [lo, hi], hi among them."""
    u = (np.arange(n) * 0.6180339887498949 + at) % 1.0
    return np.rint(lo + (hi - lo) * (u / max(u.max(), 1e-9) if n > 1 else np.ones(1))).astype(np.int64)


def sizes(c):
    """(tokens cached before the step, drafted tokens) of each sequence."""
    n = spread(c["batch"], 1 if c["drafts"] < 4 else c["drafts"] // 4, c["drafts"], 0.3) if c["drafts"] > 1 else np.ones(c["batch"], np.int64)
    return spread(c["batch"], c["lo"], c["hi"]), n


def work(c):
    if c["op"] == "lappend":
        e = c["tokens"] * (c["latent"] + c["rope"] + c["n_h"] * c["rope"])
        return {"bytes": 4 * e + 12 * c["tokens"], "flops": c["tokens"] * (4 * c["latent"] + 3 * c["rope"] * (1 + c["n_h"]))}
    base, n = sizes(c)
    if c["op"] == "accept":
        moved = int(np.ceil(n / 3).sum())
        return {"bytes": 4 * moved * c["n_kv"] * c["width"] * c["pools"], "flops": 0}
    w, v, n_kv = (c["d"], c["d"], c["n_kv"]) if c["op"] == "tree" else (c["latent"] + c["rope"], c["latent"], 1)
    rows = int((base + n).sum()) * n_kv * (2 * w if c["op"] == "tree" else w)
    io = int(n.sum()) * c["n_h"] * (2 * w + (4 if c["f32"] else 2) * v)
    return {"bytes": 2 * rows + io, "flops": 2 * (w + v) * c["n_h"] * int((n * base + n * (n + 1) // 2).sum())}


# ---- inputs -----------------------------------------------------------------------------------------
def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def tables(c, lens, r):
    """Physical blocks of each sequence, drawn from a shuffled pool a little larger than needed."""
    nb = -(-np.asarray(lens, np.int64) // c["bs"])
    blocks = int(nb.sum()) + max(1, int(nb.sum()) // 8)
    perm = r.permutation(blocks).astype(np.int32)
    bt = np.full((len(nb), max(1, int(nb.max()))), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(nb)])
    for s in range(len(nb)):
        bt[s, :nb[s]] = perm[at[s]:at[s + 1]]
    return bt, blocks


def tree(n, r):
    """Parents of n drafted tokens (-1: the sequence's last cached token): chains with branches, as drafts grow."""
    parent = np.arange(n) - 1
    branch = r.random_sample(n) < 0.5
    parent[branch] = np.floor(r.random_sample(n)[branch] * np.arange(n)[branch] * 1.2).astype(np.int64) - 1
    return np.minimum(parent, np.arange(n) - 1)


def ancestors(parent):
    """Bit j of entry i: token i attends to token j (its ancestors and itself)."""
    m = []
    for i, p in enumerate(parent):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return m


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) & 0x7fffffff)
    r = np.random.RandomState(int(seed) & 0x7fffffff)
    s, op, bs = dict(c), c["op"], c["bs"]
    dev = lambda x, t=None: torch.as_tensor(np.asarray(x) if t is None else np.asarray(x).astype(t), device=DEV)  # noqa: E731
    if op == "lappend":
        n, w, n_h, rope = c["tokens"], c["latent"] + c["rope"], c["n_h"], c["rope"]
        s["kv"] = normal(g, n, w + 64)[:, :w]                   # part of a wider projection's output
        s["q"] = normal(g, n, n_h, 128 + rope)                  # heads of a part without and a part with positions
        s["q_abs"] = normal(g, n, n_h, w)                       # the absorbed part is in place already
        s["weight"] = (1 + 0.1 * torch.randn(c["latent"], generator=g, device=DEV)).to(torch.bfloat16) if c["norm"] else None
        s["positions"] = torch.randint(0, c["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
        blocks = -(-n // bs) + 2
        s["slots"] = torch.randperm(blocks * bs, generator=g, device=DEV)[:n]
        s["cache"] = normal(g, blocks, bs, w)
        s["inv"] = torch.as_tensor(10000.0 ** (-np.arange(0, rope, 2) / rope), device=DEV)
        return s
    base, n = sizes(c)
    bt, blocks = tables(c, base + n, r)
    parents = [tree(int(k), r) for k in n]
    s["bt"], s["ctx"], s["nmax"] = dev(bt), dev(base + n, np.int32), int(n.max())
    s["start"] = dev(np.concatenate([[0], np.cumsum(n)]), np.int32)
    if op == "accept":
        path, count = np.zeros((c["batch"], s["nmax"]), np.int32), np.zeros(c["batch"], np.int32)
        for b, k in enumerate(n):                               # about a third of the tokens, one chain from the root down
            p = np.sort(r.permutation(int(k))[:-(-int(k) // 3)])
            path[b, :len(p)], count[b] = p, len(p)
        s["path"], s["count"] = dev(path), dev(count)
        shape = (blocks, bs, c["width"]) if c["n_kv"] == 1 and c["width"] > 128 else (blocks, c["n_kv"], bs, c["width"])
        s["caches"] = [normal(g, *shape) for _ in range(c["pools"])]
        return s
    T, n_h = int(n.sum()), c["n_h"]
    if c["mask"]:
        words = -(-s["nmax"] // 64)
        bits = [a >> 64 * j & (1 << 64) - 1 for p in parents for a in ancestors(p) for j in range(words)]
        s["bits"] = dev(np.array(bits, dtype=np.uint64).astype(np.int64).reshape(T, words))
    else:
        s["bits"] = None
    kind = torch.float32 if c["f32"] else torch.bfloat16
    if op == "tree":
        s["q"], s["out"] = normal(g, T, n_h, c["d"]), torch.empty(T, n_h, c["d"], dtype=kind, device=DEV)
        s["k_pool"], s["v_pool"] = normal(g, blocks, c["n_kv"], bs, c["d"]), normal(g, blocks, c["n_kv"], bs, c["d"])
        s["scale"] = c["d"] ** -0.5
        return s
    s["q"] = normal(g, T, n_h, c["latent"] + c["rope"])
    s["out"] = torch.empty(T, n_h, c["latent"], dtype=kind, device=DEV)
    s["cache"], s["scale"] = normal(g, blocks, bs, c["latent"] + c["rope"]), (c["latent"] + c["rope"]) ** -0.5
    return s


# ---- plain forms ------------------------------------------------------------------------------------
def places(s):
    """Sequence of each drafted token and its number there."""
    at = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(s["start"], at.to(torch.int32), right=True) - 1
    return seq, at - s["start"][seq]


def attention_plain(s, k, v):
    """Tokens q [T][n_h][w] over the sequences' rows k [B][n_kv][L][w] and v; drafted tokens are padded to the largest tree."""
    (B, n_kv, L, w), (T, n_h, _) = k.shape, s["q"].shape
    seq, i = places(s)
    q = torch.zeros(B, s["nmax"], n_h, w, device=DEV)
    q[seq, i] = s["q"].float()
    base = s["ctx"] - (s["start"][1:] - s["start"][:-1])
    t = torch.arange(L, device=DEV)
    j = t[None, None] - base[:, None, None]
    if s["bits"] is None:
        seen = j <= torch.arange(s["nmax"], device=DEV)[None, :, None]
    else:
        bits = torch.zeros(B, s["nmax"], s["bits"].shape[1], dtype=torch.int64, device=DEV)
        bits[seq, i] = s["bits"]
        word = (j.clamp(min=0) >> 6).clamp(max=bits.shape[2] - 1).expand(B, s["nmax"], L)
        seen = (j < 0) | ((torch.gather(bits, 2, word) >> (j.clamp(min=0) & 63)) & 1).bool()
    seen = seen & (t < s["ctx"][:, None, None])
    q = q.view(B, s["nmax"], n_kv, -1, w).permute(0, 2, 1, 3, 4).flatten(2, 3)              # [B][n_kv][token, head of the group][w]
    x = (q @ k.transpose(2, 3) * s["scale"]).view(B, n_kv, s["nmax"], -1, L)
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p / torch.where(total > 0, total, 1.0)).flatten(2, 3) @ v
    o = o.view(B, n_kv, s["nmax"], -1, v.shape[-1]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s["out"].copy_(o[seq, i])


def tree_plain(s):
    k, v = (p[s["bt"].long().clamp(min=0)].transpose(1, 2).flatten(2, 3).float() for p in (s["k_pool"], s["v_pool"]))
    attention_plain(s, k, v)


def latent_plain(s):
    k = s["cache"][s["bt"].long().clamp(min=0)].flatten(1, 2)[:, None].float()
    attention_plain(s, k, k[..., :s["latent"]])


def turn_plain(x, cos, sin, inter):
    x, h = x.float(), x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :h], x[..., h:])
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1 if inter else -2).flatten(-2).to(torch.bfloat16)


def lappend_plain(s):
    z, rope = s["latent"], s["rope"]
    ang = s["positions"].double()[:, None] * s["inv"]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    x = s["kv"][:, :z].float()
    if s["weight"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    row = torch.cat([x.to(torch.bfloat16), turn_plain(s["kv"][:, z:], cos, sin, s["inter"])], -1)
    s["cache"].view(-1, z + rope)[s["slots"]] = row
    s["q_abs"][..., z:] = turn_plain(s["q"][..., 128:], cos[:, None], sin[:, None], s["inter"])


def accept_plain(s):
    bs = s["bs"]
    base = s["ctx"] - (s["start"][1:] - s["start"][:-1])
    i = torch.arange(s["path"].shape[1], device=DEV)
    b, k = (i[None] < s["count"][:, None]).nonzero(as_tuple=True)
    to, at = base[b] + k, base[b] + s["path"][b, k]
    bt = s["bt"].long()
    place = lambda t: (bt[b, t // bs], t % bs) if s["caches"][0].dim() == 3 else (bt[b, t // bs], slice(None), t % bs)  # noqa: E731
    src, dst = place(at), place(to)
    [p.__setitem__(dst, p[src]) for p in s["caches"]]
    return (base + s["count"]).to(torch.int32)


# ---- one pass ---------------------------------------------------------------------------------------
def run_own(s):
    import paged_kv_cache_175_gb300 as pkv
    op = s["op"]
    if op == "tree":
        if "workspace" not in s:
            s["workspace"] = torch.empty(pkv.tree_workspace_bytes(s["batch"], s["q"].shape[0], s["n_h"], s["n_kv"], s["d"], s["bs"]),
                                         dtype=torch.uint8, device=DEV)
        pkv.paged_tree_attn(s["q"], s["k_pool"], s["v_pool"], s["bt"], s["ctx"], s["scale"], q_start=s["start"], tree_mask=s["bits"],
                            out=s["out"], workspace=s["workspace"])
    elif op == "latent":
        if "workspace" not in s:
            s["workspace"] = torch.empty(pkv.latent_workspace_bytes(s["batch"], s["q"].shape[0], s["n_h"], s["latent"], s["rope"], s["bs"]),
                                         dtype=torch.uint8, device=DEV)
        start = None if s["drafts"] == 1 else s["start"]
        pkv.paged_latent_attn(s["q"], s["cache"], s["latent"], s["bt"], s["ctx"], s["scale"], q_start=start, tree_mask=s["bits"],
                              out=s["out"], workspace=s["workspace"])
    elif op == "lappend":
        table = pkv.rope_table(64, s["rope"], interleaved=s["inter"])
        pkv.latent_append(s["kv"], s["q"][..., 128:], s["positions"], s["slots"], table, s["cache"], q_out=s["q_abs"][..., s["latent"]:],
                          weight=s["weight"], eps=1e-6)
    else:
        return pkv.kv_tree_accept(s["caches"], s["bt"], s["ctx"], s["start"], s["path"], s["count"])


PLAIN = {"tree": tree_plain, "latent": latent_plain, "lappend": lappend_plain, "accept": accept_plain}


def run(s):
    lens = run_own(s) if own else PLAIN[s["op"]](s)
    if s["op"] == "lappend":
        return s["q_abs"], s["cache"]
    if s["op"] == "accept":
        return lens, s["caches"]
    return s["out"]


# ---- the definitions in 64 bits ---------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "accept":
        return None                                            # rows are moved, nothing is computed
    if c["op"] == "lappend":
        z, rope, out = c["latent"], c["rope"], []
        turns = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["positions"].double()[:, None] * s["inv"])
        i = torch.arange(rope // 2, device=DEV)
        i, j = (2 * i, 2 * i + 1) if c["inter"] else (i, i + rope // 2)
        for x, by in ((s["q"][..., 128:].double(), turns[:, None]), (s["kv"][:, z:].double(), turns)):
            y, u = torch.empty_like(x), torch.complex(x[..., i], x[..., j]) * by
            y[..., i], y[..., j] = u.real, u.imag
            out.append(y)
        x = s["kv"][:, :z].double()
        if c["norm"]:
            x = x / torch.sqrt(torch.einsum("tc,tc->t", x, x) / z + 1e-6)[:, None] * s["weight"].double()
        cache = s["cache"].double()
        cache[torch.div(s["slots"], c["bs"], rounding_mode="floor"), torch.remainder(s["slots"], c["bs"])] = torch.cat([x, out[1]], 1)
        return torch.cat([s["q_abs"][..., :z].double(), out[0]], -1), cache
    base, n = sizes(c)
    at, bt, out = 0, s["bt"].long(), []
    n_kv = c["n_kv"] if c["op"] == "tree" else 1
    G = c["n_h"] // n_kv
    for b in range(c["batch"]):
        L, k = int(base[b] + n[b]), int(n[b])
        used = bt[b, :-(-L // c["bs"])]
        if c["op"] == "tree":
            K, V = (p[used].transpose(0, 1).flatten(1, 2)[:, :L] for p in (s["k_pool"], s["v_pool"]))
        else:
            K = s["cache"][used].flatten(0, 1)[None, :L]
            V = K[..., :c["latent"]]
        see = torch.zeros(k, L, dtype=torch.bool, device=DEV)
        see[:, :L - k] = True
        if c["mask"]:
            words = s["bits"][at:at + k].cpu().numpy().astype(np.uint64)
            for a in range(k):
                see[:, L - k + a] = torch.as_tensor((words[:, a // 64] >> np.uint64(a % 64)) & np.uint64(1) != 0, device=DEV)
        else:
            see[:, L - k:] = torch.ones(k, k, device=DEV).tril() > 0
        o = []
        for g in range(n_kv):
            q = s["q"][at:at + k, g * G:(g + 1) * G].double().transpose(0, 1)                # [head][token][w]
            x = torch.where(see, torch.einsum("hiw,tw->hit", q, K[g].double()) * s["scale"], -math.inf)
            o.append(torch.einsum("hit,tv->hiv", torch.softmax(x, -1), V[g].double()))
        out.append(torch.cat(o).transpose(0, 1))
        at += k
    return torch.cat(out)
