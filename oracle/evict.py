"""Accounted attention and eviction by accumulated attention weight.  Test infrastructure only.

Every cached token's account grows by the attention weight it gets from the query heads of its kv
group at each step.  An eviction to a budget of K rows keeps, per kv head, those of the sequence's
last `recent` tokens that are still held, and those with the largest accounts (ties: lowest row); kept rows below K stay in place and
the kept rows at or behind K fill the rows below K that were dropped, both in ascending order.
"""
import numpy as np

from .paged_attention import attention_weights, gather_sequence


def attention_mass(q, k_pool, block_tables, context_lens, scale, block_size, width):
    """[B][n_kv][width] float64: sum over the group's heads of the softmax weights; 0 behind the context."""
    q = np.asarray(q, dtype=np.float64)
    B, n_h, _ = q.shape
    n_kv = k_pool.shape[1]
    G = n_h // n_kv
    out = np.zeros((B, n_kv, width))
    for s in range(B):
        L = int(context_lens[s])
        for g in range(n_kv if L > 0 else 0):
            K = gather_sequence(k_pool, block_tables[s], L, g, block_size)
            for h in range(g * G, (g + 1) * G):
                out[s, g, :L] += attention_weights(q[s, h], K, scale)
    return out


def evict_rows(mass, positions, n, K, recent, seen):
    """(holes, movers) of one (sequence, kv head): rows below K that go, rows behind that replace them.
    positions: the token each of the n rows holds, of the `seen` that the sequence had."""
    newest = seen - 1
    recent = min(recent, K)
    def rank(r):
        m = mass[r]
        m = np.inf if np.isnan(m) else m
        return (0 if positions[r] > newest - recent else 1, 0 if np.isnan(mass[r]) else 1, -m,
                0 if not np.signbit(mass[r]) else 1, r)
    stay = set(sorted(range(n), key=rank)[:K])
    return [r for r in range(K) if r not in stay], [r for r in range(K, n) if r in stay]


def evict(k_pool, v_pool, block_tables, context_lens, keep, recent, mass, positions, kept, dropped, block_size):
    """New (k_pool, v_pool, mass, positions, kept, dropped, new_lens); inputs are left as they are."""
    kp, vp, mass, positions, kept, dropped = (np.array(x, copy=True) for x in (k_pool, v_pool, mass, positions, kept, dropped))
    new = np.array(context_lens, copy=True)
    src_mass = mass.copy()
    for s in range(len(context_lens)):
        n, K = int(context_lens[s]), max(0, min(int(keep[s]), int(context_lens[s])))
        new[s] = K
        if K == n:
            continue
        for g in range(mass.shape[1]):
            pos = np.array([positions[s, g, r] if r < kept[s] else dropped[s] + r for r in range(n)])
            holes, movers = evict_rows(src_mass[s, g], pos, n, K, recent, dropped[s] + n)
            at = lambda r: (int(block_tables[s, r // block_size]), g, r % block_size)
            for h, m in zip(holes, movers):
                kp[at(h)], vp[at(h)] = k_pool[at(m)], v_pool[at(m)]
                mass[s, g, h], pos[h] = src_mass[s, g, m], pos[m]
            mass[s, g, K:n] = 0
            positions[s, g, :K] = pos[:K]
        kept[s], dropped[s] = K, dropped[s] + n - K
    return kp, vp, mass, positions, kept, dropped, new
