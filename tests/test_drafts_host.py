"""Drafted tokens and the latent cache without a GPU: pins of the oracle, refusals of the C calls and the binding."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_175_gb300 as pkv
from oracle import drafts as od
from paged_kv_cache_175_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_library()


def rows(rng, B, n_kv, L, w):
    x = rng.normal(size=(B, n_kv, L, w))
    return x, lambda s: x[s]


def test_chain_is_one_decode_step_after_another():
    rng = np.random.default_rng(0)
    L, n = 20, 6
    K, keys = rows(rng, 1, 2, L, 8)
    V, values = rows(rng, 1, 2, L, 8)
    q = rng.normal(size=(n, 4, 8))
    out, _ = od.step_attention(q, keys, values, [0, n], [L], 0.3)
    for i in range(n):
        t = L - n + i + 1
        for h in range(4):
            assert np.allclose(out[i, h], oracle.attention_weights(q[i, h], K[0, h // 2, :t], 0.3) @ V[0, h // 2, :t], atol=1e-13)


def test_tree_is_the_chains_of_its_paths():
    rng = np.random.default_rng(1)
    L, parents = 15, [-1, 0, 0, 2, 1]
    anc = []
    for i, p in enumerate(parents):
        anc.append((anc[p] if p >= 0 else 0) | 1 << i)
    K, keys = rows(rng, 1, 1, L, 4)
    V, values = rows(rng, 1, 1, L, 4)
    q = rng.normal(size=(5, 2, 4))
    out, _ = od.step_attention(q, keys, values, [0, 5], [L], 1.0, np.array(anc, np.int64)[:, None])
    for path in ([0, 1, 4], [0, 2, 3]):
        keep = list(range(10)) + [10 + p for p in path]
        K2, V2 = K[:, :, keep], V[:, :, keep]
        o, _ = od.step_attention(q[path], lambda s: K2[s], lambda s: V2[s], [0, 3], [13], 1.0)
        assert np.allclose(out[path], o, atol=1e-13)


def test_nothing_attended_gives_zeros_and_words_end_the_mask():
    rng = np.random.default_rng(2)
    _, keys = rows(rng, 1, 1, 70, 4)
    q = rng.normal(size=(70, 1, 4))
    mask = np.zeros((70, 1), np.int64)
    mask[3] = -1
    out, size = od.step_attention(q, keys, keys, [0, 70], [70], 1.0, mask)
    assert not out[[0, 1, 2]].any() and not out[4:].any()
    assert od.seen(70, mask)[3].sum() == 64


def test_accept_moves_the_path_and_nothing_else():
    rng = np.random.default_rng(3)
    pool, table = rng.normal(size=(6, 2, 4, 3)), [5, 1, 3]
    out, n = od.accept(pool, table, 11, 6, [1, 2, 5], 4)         # rows 5.. hold the six tokens
    row = lambda p, t: p[table[t // 4], :, t % 4]  # noqa: E731
    assert n == 8
    for t, src in [(i, i) for i in range(5)] + [(5, 6), (6, 7), (7, 10)] + [(i, i) for i in (8, 9, 10)]:
        assert np.array_equal(row(out, t), row(pool, src))
    assert np.array_equal(out[[0, 2, 4]], pool[[0, 2, 4]])


def test_latent_rows_have_norm_one_and_keep_relative_angles():
    rng = np.random.default_rng(4)
    kv = rng.normal(size=(2, 256 + 32))
    f, a = oracle.rope_frequencies(32)
    r = od.latent_rows(kv, 256, [7, 900], f, a, False, np.ones(256), 0.0)
    assert np.allclose((r[:, :256] ** 2).mean(1), 1.0)
    s = od.latent_rows(kv, 256, [107, 1000], f, a, False)
    assert np.allclose(s[:, :256], kv[:, :256])
    assert np.isclose(r[0, 256:] @ r[1, 256:], s[0, 256:] @ s[1, 256:])


# ---- refusals -----------------------------------------------------------------------------------------
P = ctypes.c_void_p(4096)                                      # an aligned address: refusals come before any use


def tree(**k):
    a = dict(q=P, k=P, v=P, bt=P, mb=4, ctx=P, start=None, mask=None, words=0, scale=1.0, T=6, B=3, n_h=8, n_kv=2, d=128, bs=16, nb=9,
             out=P, kind=0, ws=P, ws_bytes=1 << 40, err=None, stream=None) | k
    return pkv.lib().pkv_paged_tree_attn(*a.values())


def latent(**k):
    a = dict(q=P, cache=P, bt=P, mb=4, ctx=P, start=None, mask=None, words=0, scale=1.0, T=6, B=3, n_h=8, latent=512, rope=64, bs=16, nb=9,
             out=P, kind=0, ws=P, ws_bytes=1 << 40, err=None, stream=None) | k
    return pkv.lib().pkv_paged_latent_attn(*a.values())


def append(**k):
    t = pkv.rope_table(64, k.pop("rot", 64))
    a = dict(kv=P, ks=576, q=P, qs=8 * 64, qh=64, pos=P, slots=P, n=3, table=ctypes.byref(t), weight=P, eps=1e-6, out=P, os=8 * 64, oh=64, cache=P,
             nb=9, bs=16, n_h=8, latent=512, rope=64, err=None, stream=None) | k
    return pkv.lib().pkv_latent_append(*a.values())


def accept(**k):
    arr = (ctypes.c_void_p * 2)(4096, 8192)
    a = dict(caches=arr, n=2, rb=256, heads=2, bt=P, mb=4, ctx=P, start=None, T=6, path=P, ps=4, count=P, lens=ctypes.c_void_p(1 << 20), B=3, bs=16, nb=9,
             err=None, stream=None) | k
    return pkv.lib().pkv_kv_tree_accept(*a.values())


EINVAL, ERANGE = -1, -2
BIG = 0x7fffffff


@pytest.mark.parametrize("call,bad", [
    (tree, dict(d=96)), (tree, dict(bs=8)), (tree, dict(n_h=7)), (tree, dict(n_h=130)), (tree, dict(n_kv=0)), (tree, dict(B=4)),
    (tree, dict(T=-1)), (tree, dict(B=-1)), (tree, dict(mb=-1)), (tree, dict(nb=-1)), (tree, dict(kind=2)), (tree, dict(mask=P)),
    (tree, dict(q=None)), (tree, dict(v=None)), (tree, dict(out=None)), (tree, dict(ws=None)), (tree, dict(ctx=None)), (tree, dict(bt=None)),
    (tree, dict(q=ctypes.c_void_p(4104))), (tree, dict(ws=ctypes.c_void_p(4096 + 16))), (tree, dict(mask=ctypes.c_void_p(4100), words=1)),
    (latent, dict(latent=384)), (latent, dict(rope=16)), (latent, dict(n_h=1025)), (latent, dict(n_h=0)), (latent, dict(B=4)), (latent, dict(bs=48)),
    (latent, dict(cache=None)), (latent, dict(cache=ctypes.c_void_p(4104))), (latent, dict(kind=-1)), (latent, dict(mask=P)),
    (append, dict(rot=32)), (append, dict(latent=128)), (append, dict(rope=16)), (append, dict(bs=24)), (append, dict(n=-1)), (append, dict(n_h=0)),
    (append, dict(n_h=1025)), (append, dict(ks=568)), (append, dict(ks=580)), (append, dict(qh=56)), (append, dict(qs=500)), (append, dict(os=504)),
    (append, dict(eps=-1.0)), (append, dict(eps=float("nan"))), (append, dict(table=None)), (append, dict(cache=None)), (append, dict(kv=ctypes.c_void_p(4104))),
    (append, dict(weight=ctypes.c_void_p(4104))), (append, dict(out=ctypes.c_void_p(4104))),
    (accept, dict(n=0)), (accept, dict(rb=24)), (accept, dict(rb=0)), (accept, dict(heads=0)), (accept, dict(T=7)), (accept, dict(B=-1)),
    (accept, dict(bs=20)), (accept, dict(path=None)), (accept, dict(count=None)), (accept, dict(lens=None)), (accept, dict(lens=P)), (accept, dict(caches=None)),
    (accept, dict(caches=(ctypes.c_void_p * 2)(4096, None))), (accept, dict(caches=(ctypes.c_void_p * 2)(4096, 4104))), (accept, dict(ps=-1)),
], ids=lambda x: x.__name__ if callable(x) else "-".join(x))
def test_arguments_are_refused(call, bad):
    assert call(**bad) == EINVAL


def test_ranges_and_empty_calls():
    assert tree(mb=0x7fff0000 // 16 + 1) == ERANGE and latent(mb=0x7fff0000 // 64 + 1, bs=64) == ERANGE
    assert accept(mb=0x7fff0000 // 16 + 1) == ERANGE
    assert tree(T=3 * (BIG // 16), n_h=64, n_kv=8) == ERANGE
    assert tree(T=0) == 0 and tree(T=0, B=0, q=None, ws=None) == 0 and latent(T=0) == 0 and append(n=0, kv=None) == 0 and accept(B=0, bt=None) == 0
    assert pkv.lib().pkv_tree_workspace_bytes(1, 1, 7, 2, 128, 16) == 0 and pkv.lib().pkv_latent_workspace_bytes(1, 1, 7, 100, 64, 16) == 0
    for w in (pkv.tree_workspace_bytes, pkv.latent_workspace_bytes):
        with pytest.raises(pkv.PkvError):
            w(-1, 1, 8, 2, 128, 16)


def test_binding_refuses_cpu_tensors():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    i32, bt, ctx = torch.int32, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: pkv.paged_tree_attn(z(2, 4, 64), z(3, 2, 16, 64), z(3, 2, 16, 64), bt, ctx, 1.0),
                 lambda: pkv.paged_latent_attn(z(2, 4, 576), z(3, 16, 576), 512, bt, ctx, 1.0),
                 lambda: pkv.latent_append(z(2, 576), z(2, 4, 64), ctx, ctx.long(), pkv.rope_table(64), z(3, 16, 576)),
                 lambda: pkv.kv_tree_accept([z(3, 2, 16, 64)], bt, ctx, z(3, t=i32), bt, ctx),
                 lambda: pkv.kv_tree_accept([z(3, 2, 16, 64)], bt, ctx, None, bt, ctx)):
        with pytest.raises(pkv.PkvError):
            call()
