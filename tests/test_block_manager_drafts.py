"""The block manager's side of drafted tokens: their rows are nobody else's, whatever tokens they hold, until a path is
accepted; then the path's tokens, in its order, are what the tree knows.  Host code only (no GPU)."""
import re

import numpy as np
import pytest

import oracle
import paged_kv_cache_175_gb300 as pkv
from oracle import drafts as od

BS = 4


def prefix(tokens):
    """What a cached row holds, by the tokens up to it."""
    return hash(tuple(int(t) for t in tokens)) & 0x7fffffff


def test_drafted_rows_are_not_reused():
    for m in (pkv.BlockManager(16, BS), oracle.BlockManager(16, BS)):
        m.add_sequence(1, [1, 2, 3, 4, 5])
        m.append_drafts([1], [7])                              # tokens 6 .. 12, say, of which all blocks are full
        assert m.add_sequence(2, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13])[1] == 4
        m.accept_drafts([1], [[6, 9, 10]])                     # rows now hold 5 6 9 10
        assert m.add_sequence(3, [1, 2, 3, 4, 5, 6, 9, 10, 11])[1] == 8
        assert m.add_sequence(4, [1, 2, 3, 4, 5, 6, 7, 8, 9])[1] == 8      # sequence 2's own


def test_rejected_blocks_are_given_back_and_shared_prompts_stay():
    m = pkv.BlockManager(12, BS)
    prompt = list(range(9))
    m.add_sequence(1, prompt)
    m.add_sequence(2, prompt)                                  # shares two blocks
    before = m.counts()["free"]
    slots = m.append_drafts([1, 2], [10, 3])
    t, lens = m.tables([1, 2], 5)
    assert lens.tolist() == [19, 12] and slots.dtype == np.int64
    where = [t[s][r // BS] * BS + r % BS for s, rows in ((0, range(9, 19)), (1, range(9, 12))) for r in rows]
    assert slots.tolist() == where
    m.accept_drafts([1, 2], [[9, 20], []])
    t, lens = m.tables([1, 2], 5)
    assert lens.tolist() == [11, 9] and (t[:, 3:] == -1).all() and m.counts()["free"] == before
    assert m.append_tokens([1], [21]).tolist() == [t[0][2] * BS + 3]       # row 11, the last of its block
    m.release(1)
    assert m.add_sequence(3, prompt + [20, 21, 0, 0])[1] == 8              # 9 0? no: that block holds 8 9 20 21
    assert m.add_sequence(4, prompt + [9, 20, 21, 0])[1] == 12


def test_refusals_change_nothing():
    m = pkv.BlockManager(4, BS)
    m.add_sequence(1, [1, 2, 3, 4, 5])
    m.add_sequence(2, [6])
    for call in (lambda: m.append_drafts([1, 9], [2, 2]), lambda: m.append_drafts([1, 1], [2, 2]), lambda: m.append_drafts([1], [-1]),
                 lambda: m.append_drafts([1, 2], [2, 9]), lambda: m.append_drafts([1], [0x7fffffff]), lambda: m.append_drafts([1, 2], [2]),
                 lambda: m.accept_drafts([1], [[3]]), lambda: m.accept_drafts([9], [[]]), lambda: m.accept_drafts([1, 2], [[]])):
        with pytest.raises(pkv.PkvError):
            call()
        t, lens = m.tables([1, 2], 2)
        assert lens.tolist() == [5, 1] and (t >= 0).sum() == 3 and m.counts()["free"] == 1
    m.append_drafts([1, 2], [3, 3])
    for call in (lambda: m.append_drafts([1], [1]), lambda: m.append_tokens([1], [6]), lambda: m.evict(1, 4), lambda: m.slide_window(1, 1),
                 lambda: m.accept_drafts([1], [[6, 7, 8, 9]]), lambda: m.accept_drafts([1, 2, 1], [[6], [7], []])):
        with pytest.raises(pkv.PkvError):
            call()
        assert m.tables([1, 2], 2)[1].tolist() == [8, 4]
    m.accept_drafts([2], [[7, 8, 9]])
    m.release(1)                                               # drafts that nothing was accepted of
    assert m.counts()["free"] == 2 and m.counts()["cached"] == 1
    assert m.append_drafts([2], [0]).size == 0
    m.accept_drafts([2], [[]])


def test_a_sequence_that_slid_its_window():
    # it holds a few of the pool's blocks, of a line that is longer than the pool
    for m in (pkv.BlockManager(4, BS), oracle.BlockManager(4, BS)):
        m.add_sequence(1, [1])
        for i in range(40):
            m.slide_window(1, 3)
            (m.append_tokens([1], [i]) if isinstance(m, pkv.BlockManager) else m.append_token(1, i))
        assert len(m.append_drafts([1], [6])) == 6
        with pytest.raises((pkv.PkvError, ValueError)):
            m.slide_window(1, 3)
        m.accept_drafts([1], [[8, 9]])


@pytest.mark.parametrize("seed", range(8))
def test_random_steps_keep_rows_and_match_the_oracle(seed):
    """Requests that share prompts, decode, draft trees and accept paths: the native manager does what the oracle does, and every row
    of a running sequence, the reused ones among them, holds what its tokens say."""
    rng = np.random.default_rng(seed)
    N, H = 40, 10
    ref, nat = oracle.BlockManager(N, BS, host_blocks=H), pkv.BlockManager(N, BS, host_blocks=H)
    pool, host = np.full((N, 1, BS, 1), -1, np.int64), np.full((H, 1, BS, 1), -1, np.int64)
    prompts = [list(rng.integers(0, 4, size=int(rng.integers(BS, 3 * BS)))) for _ in range(4)]
    live, sid, reused, drafted = {}, 0, 0, 0

    def both(f, *a):
        got = want = None
        try:
            want = f(ref, *a)
        except (oracle.OutOfBlocks, ValueError):
            want = "refused"
        try:
            got = f(nat, *a)
        except pkv.PkvError:
            got = "refused"
        same = np.array_equal(got, want) if isinstance(got, np.ndarray) else got == want
        assert same, (seed, got, want)
        c, copies = ref.take_copies(), nat.take_copies().tolist()
        assert copies == [list(x) for x in c]
        oracle.apply_copies(c, pool, host)
        return got

    def write(s, t, value):
        b, _ = ref.table(s)
        pool[b[t // BS], 0, t % BS, 0] = value

    for _ in range(300):
        op = rng.random()
        if op < 0.25 or not live:
            sid += 1
            toks = prompts[int(rng.integers(4))] + [int(x) for x in rng.integers(0, 4, size=int(rng.integers(0, 2 * BS)))]
            got = both(lambda m: m.add_sequence(sid, toks))
            if got != "refused":
                live[sid] = list(toks)
                reused += got[1]
                for t in range(got[1], len(toks)):
                    write(sid, t, prefix(toks[:t + 1]))
        elif op < 0.5:
            s, x = int(rng.choice(list(live))), int(rng.integers(0, 4))
            one = lambda m: m.append_token(s, x) if m is ref else int(m.append_tokens([s], [x])[0])  # noqa: E731
            if both(one) != "refused":
                live[s].append(x)
                write(s, len(live[s]) - 1, prefix(live[s]))
        elif op < 0.85:
            s, n = int(rng.choice(list(live))), int(rng.integers(1, 11))
            if isinstance(both(lambda m: np.asarray(m.append_drafts([s], [n]))), str):
                continue
            drafted += n
            base = len(live[s])
            parent = [int(rng.integers(-1, i)) if i else -1 for i in range(n)]
            tok = [int(x) for x in rng.integers(0, 4, size=n)]
            chain = [[]]
            for i in range(n):
                chain.append((chain[parent[i] + 1] if parent[i] >= 0 else []) + [i])
                write(s, base + i, prefix(live[s] + [tok[j] for j in chain[-1]]))
            path = chain[int(rng.integers(0, n + 1))]
            if rng.random() < 0.3:                             # another request in between, with the drafts in their order
                sid += 1
                toks = live[s] + tok + [0]
                got = both(lambda m: m.add_sequence(sid, toks))
                if got != "refused":
                    live[sid] = list(toks)
                    reused += got[1]
                    for t in range(got[1], len(toks)):
                        write(sid, t, prefix(toks[:t + 1]))
            table, lens = nat.tables([s], N)
            assert lens[0] == base + n
            pool[:] = od.accept(pool, table[0], lens[0], n, path, BS)[0].astype(np.int64)
            both(lambda m: m.accept_drafts([s], [[tok[j] for j in path]]))
            live[s] += [tok[j] for j in path]
        else:
            s = int(rng.choice(list(live)))
            both(lambda m: m.release(s))
            del live[s]
        for s, toks in live.items():
            table, lens = nat.tables([s], N)
            assert lens[0] == len(toks)
            rows = [int(pool[table[0][t // BS], 0, t % BS, 0]) for t in range(len(toks))]
            assert rows == [prefix(toks[:t + 1]) for t in range(len(toks))], (seed, s)
        c, r = nat.counts(), ref.counts()
        assert (c["free"], c["active"], c["cached"], c["host"]) == (r["free"], r["active"], r["cached"], r["host"])
    assert reused > 50 and drafted > 100


def test_the_readme_shows_them():
    text = open(__file__.replace("tests/test_block_manager_drafts.py", "README.md")).read()
    code = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "append_drafts" in b]
    assert len(code) == 1
    calls = []
    manager = pkv.BlockManager(32, BS)
    manager.add_sequence(7, [1, 2, 3, 4, 5])
    manager.add_sequence(8, [1, 2, 3, 4])

    class Calls:
        def __getattr__(self, name):
            return lambda *a, **k: calls.append(name)

    path, n_accept = np.array([[0, 2, 9], [1, 0, 0]]), np.array([2, 1])
    exec(code[0], dict(manager=manager, pkv=Calls(), sequences=[7, 8], drafted=[[10, 11, 12], [20, 21]], max_blocks=4, path=path, n_accept=n_accept,
                       **{n: None for n in ("caches", "q_start", "device_path", "device_n_accept")}, device=lambda x: x))
    assert calls == ["kv_tree_accept"]
    assert manager.tables([7, 8], 4)[1].tolist() == [7, 5]
    manager.append_tokens([7], [13])
    assert manager.add_sequence(9, [1, 2, 3, 4, 5, 10, 12, 13, 0])[1] == 8
