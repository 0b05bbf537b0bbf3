"""Every tensor argument of the serving calls is checked before anything runs: type, device, shape, layout."""
import threading

import pytest
import torch

import paged_kv_cache_175_gb300 as pkv

pytestmark = pytest.mark.gpu
B, NH, NKV, D, BS, NB, MB, T = 3, 4, 2, 64, 16, 8, 2, 32


def rnd(*shape):
    return torch.randn(*shape, device="cuda").bfloat16()


def ints(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def rope_append(**k):
    a = dict(q=rnd(B, NH, D), k=rnd(B, NKV, D), v=rnd(B, NKV, D), positions=ints(B), slot_mapping=torch.arange(B, device="cuda"),
             k_pool=rnd(NB, NKV, BS, D), v_pool=rnd(NB, NKV, BS, D), q_out=rnd(B, NH, D), err=ints(1)) | k
    return a, lambda: pkv.rope_append(table=pkv.rope_table(D), **a)


def rope_qk(**k):
    a = dict(q=rnd(B, NH, D), k=rnd(B, NKV, D), positions=ints(B), q_out=rnd(B, NH, D), k_out=rnd(B, NKV, D)) | k
    return a, lambda: pkv.rope_qk(table=pkv.rope_table(D), **a)


def cache_of(a):
    return pkv.Q8CacheTensors(a["records"], a["k_tail"], a["v_tail"])


def q8_tensors():
    c = pkv.alloc_q8_cache(NB, NKV, BS, D, B)
    return dict(records=c.records, k_tail=c.k_tail, v_tail=c.v_tail)


def without(a, *names):
    return {n: t for n, t in a.items() if n not in names}


def append_q8(**k):
    a = dict(k=rnd(B, NKV, D), v=rnd(B, NKV, D), slot_mapping=torch.arange(B, device="cuda") * BS,
             tail_seq=torch.arange(B, dtype=torch.int32, device="cuda"), err=ints(1), **q8_tensors()) | k
    return a, lambda: pkv.kv_quant_append_q8(cache=cache_of(a), **without(a, "records", "k_tail", "v_tail"))


def attn_q8(**k):
    a = dict(q=rnd(B, NH, D), block_tables=ints(B, MB), context_lens=ints(B) + 16, out=rnd(B, NH, D),
             workspace=torch.empty(pkv.q8_workspace_bytes(B, NH, NKV, D, BS), dtype=torch.uint8, device="cuda"), err=ints(1),
             **q8_tensors()) | k
    return a, lambda: pkv.paged_decode_attn_q8(cache=cache_of(a), scale=0.125, **without(a, "records", "k_tail", "v_tail"))


def attn_mass(**k):
    a = dict(q=rnd(B, NH, D), k_pool=rnd(NB, NKV, BS, D), v_pool=rnd(NB, NKV, BS, D), block_tables=ints(B, MB),
             context_lens=ints(B) + 16, mass=torch.zeros(B, NKV, T, device="cuda"), out=rnd(B, NH, D),
             workspace=torch.empty(pkv.mass_workspace_bytes(B, NH, NKV, D, BS, MB), dtype=torch.uint8, device="cuda"),
             err=ints(1)) | k
    return a, lambda: pkv.paged_decode_attn_mass(scale=0.125, **a)


def evict(**k):
    st = pkv.alloc_evict_state(B, NKV, T)
    tables = torch.arange(B * MB, dtype=torch.int32, device="cuda").reshape(B, MB)
    a = dict(k_pool=rnd(NB, NKV, BS, D), v_pool=rnd(NB, NKV, BS, D), block_tables=tables, context_lens=ints(B) + 20,
             keep=ints(B) + 16, new_lens=ints(B), mass=st.mass, positions=st.positions, kept=st.kept, dropped=st.dropped,
             workspace=torch.empty(pkv.evict_workspace_bytes(B, NKV, BS, MB), dtype=torch.uint8, device="cuda"), err=ints(1)) | k
    names = ("mass", "positions", "kept", "dropped")
    return a, lambda: pkv.kv_evict(recent=4, state=pkv.EvictState(*(a[n] for n in names)), **without(a, *names))


CALLS = (rope_append, rope_qk, append_q8, attn_q8, attn_mass, evict)
STRIDED_TOKENS = ("q", "k", "v", "q_out", "k_out")           # of the rotary calls and the append


def wrong(t, name):
    yield "device", t.cpu()
    if name != "workspace":
        yield "type", t.to(torch.float16 if t.is_floating_point() else torch.int16)
    if name not in ("err", "workspace"):
        yield "dims", t[None]
        if t.numel() > 1:
            yield "size", torch.cat([t, t[..., :1]], -1)      # one more of the last dimension
            wide = torch.cat([t, t], -1)                      # the same shape, a gap after every row
            yield "layout", wide[..., ::2] if t.dim() == 1 or name in STRIDED_TOKENS else wide[..., :t.shape[-1]]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_every_tensor_is_checked(call):
    args, run = call()
    run()                                                      # as given, it is taken
    for name, t in args.items():
        for what, bad in wrong(t, name):
            if what == "size" and (name == "block_tables" or (name == "mass" and call is attn_mass)):
                continue                                       # wider accounts and tables are other valid sizes
            with pytest.raises((pkv.PkvError, ValueError)):
                call(**{name: bad})[1]()
                pytest.fail(f"{name}: {what} was taken")
    torch.cuda.synchronize()
    run()


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_parameters_are_tensors(call):
    args, _ = call()
    cast = {n: torch.nn.Parameter(t, requires_grad=False) for n, t in args.items()}
    call(**cast)[1]()
    torch.cuda.synchronize()


def test_numbers_are_checked():
    c = pkv.alloc_q8_cache(NB, NKV, BS, D, B)
    q, bt, ctx = rnd(B, NH, D), ints(B, MB), ints(B) + 16
    for kw in (dict(window=-1), dict(window=1 << 40), dict(scale="x"), dict(scale=None)):
        with pytest.raises(pkv.PkvError):
            pkv.paged_decode_attn_q8(q, c, bt, ctx, **{**dict(scale=1.0), **kw})
    st = pkv.alloc_evict_state(B, NKV, T)
    for recent in (-1, 1 << 40):
        with pytest.raises(pkv.PkvError):
            pkv.kv_evict(rnd(NB, NKV, BS, D), rnd(NB, NKV, BS, D), bt, ctx, ctx, recent, st)
    torch.cuda.synchronize()


def test_calls_from_two_threads():
    """Two threads on streams of their own: each gets the result of its own arguments."""
    table = pkv.rope_table(D)
    ins = [(rnd(64, NH, D), rnd(64, NKV, D), torch.arange(64, dtype=torch.int32, device="cuda") + 7 * i) for i in range(2)]
    want = [pkv.rope_qk(*x, table) for x in ins]
    torch.cuda.synchronize()
    got, fails = [None, None], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[i] = [pkv.rope_qk(*ins[i], table) for _ in range(50)]
            s.synchronize()
        except Exception as e:                                 # noqa: BLE001
            fails.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not fails
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y[0], want[i][0]) and torch.equal(y[1], want[i][1])
