"""Drafted tokens and the latent cache, restated plainly in float64 (test infrastructure only).

* Attention of several tokens per sequence: token i of a sequence with n drafted tokens (its last n cached
  rows) attends to every row before them and, of them, to those its mask names (no mask: up to itself).
  One row per (token, head); nothing attended gives zeros.
* The latent cache: one vector per token for all heads; keys are the vectors, values their first `latent`
  channels.
* Acceptance: the rows of an ascending path move to the front of the drafted ones.
"""
import numpy as np

from .rope import rope_tokens


def seen(n, mask=None):
    """bool [n][n]: which drafted tokens each one attends to.  mask: int64 words [n][words]."""
    if mask is None:
        return np.tril(np.ones((n, n), dtype=bool))
    out = np.zeros((n, n), dtype=bool)
    for i in range(n):
        for j in range(min(n, 64 * mask.shape[1])):
            out[i, j] = (int(mask[i, j // 64]) >> (j % 64)) & 1
    return out


def step_attention(q, keys, values, starts, context_lens, scale, masks=None):
    """q [T][n_h][w]; keys(s) / values(s): [n_kv][ctx][.] of sequence s.  Returns (out [T][n_h][v], |p| |v| sums of
    the same shape) in float64; rows of tokens in no sequence are NaN."""
    T, n_h, _ = q.shape
    out = size = None
    for s in range(len(context_lens)):
        L, a, b = int(context_lens[s]), int(starts[s]), int(starts[s + 1])
        K, V = keys(s), values(s)
        G = n_h // K.shape[0]
        if out is None:
            out = np.full((T, n_h, V.shape[2]), np.nan)
            size = np.zeros_like(out)
        n = b - a
        see = seen(n, None if masks is None else masks[a:b])
        for i in range(n):
            rows = [t for t in range(min(L, L - n))] if L > n else []
            rows += [L - n + j for j in range(n) if see[i, j] and L - n + j >= 0]
            for h in range(n_h):
                if not rows or L <= 0:
                    out[a + i, h] = 0.0
                    continue
                x = scale * (K[h // G][rows] @ q[a + i, h])
                p = np.exp(x - x.max())
                p /= p.sum()
                out[a + i, h] = p @ V[h // G][rows]
                size[a + i, h] = p @ np.abs(V[h // G][rows])
    return out, size


def paged(pool, table, ctx, bs):
    """Rows 0..ctx-1 of a sequence: pool [num_blocks][heads][bs][w] -> [heads][ctx][w]."""
    w = pool.shape[-1]
    if ctx <= 0:
        return np.zeros((pool.shape[1], 0, w))
    blocks = [pool[int(b)] for b in table[:-(-int(ctx) // bs)]]
    return np.concatenate(blocks, axis=1)[:, :int(ctx)].astype(np.float64)


def latent_rows(kv, latent, positions, freqs, amp, interleaved, weight=None, eps=1e-6):
    """Vectors as they are cached: [n][latent + rope]."""
    c, k = kv[:, :latent], kv[:, latent:]
    if weight is not None:
        c = c / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps) * weight
    return np.concatenate([c, rope_tokens(k[:, None], positions, freqs, amp, interleaved=interleaved)[:, 0]], axis=1)


def accept(pool, table, ctx, n, path, bs):
    """(pool after the moves, new length) of one sequence; pool [num_blocks][heads][bs][w]."""
    out, base, done = np.array(pool, copy=True), int(ctx) - int(n), 0
    if base < 0:
        return out, int(ctx)
    for i, p in enumerate(path):
        if p <= (path[i - 1] if i else -1) or p >= n:
            break
        a, b = base + int(p), base + i
        out[table[b // bs], :, b % bs] = pool[table[a // bs], :, a % bs]
        done += 1
    return out, base + done
