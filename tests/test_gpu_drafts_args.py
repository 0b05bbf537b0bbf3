"""Calls for drafted tokens and for the latent cache: every tensor argument is checked before anything runs, buffers on
streams of their own are safe, and calls from two threads get their own results."""
import threading

import pytest
import torch

import paged_kv_cache_175_gb300 as pkv
from test_gpu_serving_args import ints, rnd, wrong
from test_gpu_side_streams import SLEEP, freed_under_way

pytestmark = pytest.mark.gpu
B, T, NH, NKV, D, LAT, ROPE, BS, NB, MB = 3, 7, 4, 2, 64, 256, 32, 16, 12, 3
TABLES = torch.arange(B * MB, dtype=torch.int32).reshape(B, MB)
STARTS = torch.tensor([0, 2, 3, 7], dtype=torch.int32)


def step(**k):
    return dict(block_tables=TABLES.cuda(), context_lens=ints(B) + 40, q_start=STARTS.cuda(),
                tree_mask=torch.full((T, 1), 3, dtype=torch.int64, device="cuda"), err=ints(1)) | k


def tree(**k):
    a = dict(q=rnd(T, NH, D), k_pool=rnd(NB, NKV, BS, D), v_pool=rnd(NB, NKV, BS, D), out=rnd(T, NH, D),
             workspace=torch.empty(pkv.tree_workspace_bytes(B, T, NH, NKV, D, BS), dtype=torch.uint8, device="cuda"), **step()) | k
    return a, lambda **kw: pkv.paged_tree_attn(scale=0.125, **a, **kw)


def latent(**k):
    a = dict(q=rnd(T, NH, LAT + ROPE), cache=rnd(NB, BS, LAT + ROPE), out=rnd(T, NH, LAT),
             workspace=torch.empty(pkv.latent_workspace_bytes(B, T, NH, LAT, ROPE, BS), dtype=torch.uint8, device="cuda"), **step()) | k
    return a, lambda **kw: pkv.paged_latent_attn(latent=LAT, scale=0.0625, **a, **kw)


def append(**k):
    a = dict(kv=rnd(T, LAT + ROPE), q=rnd(T, NH, ROPE), positions=ints(T) + 5, slot_mapping=torch.arange(T, device="cuda"),
             cache=rnd(NB, BS, LAT + ROPE), q_out=rnd(T, NH, ROPE), weight=rnd(LAT), err=ints(1)) | k
    return a, lambda **kw: pkv.latent_append(table=pkv.rope_table(64, ROPE), **a, **kw)


def accept(**k):
    a = dict(block_tables=TABLES.cuda(), context_lens=ints(B) + 40, q_start=STARTS.cuda(),
             path=torch.tensor([[0, 1], [0, 0], [1, 3]], dtype=torch.int32, device="cuda"),
             n_accept=torch.tensor([2, 1, 2], dtype=torch.int32, device="cuda"), new_lens=ints(B), err=ints(1)) | k
    return a, lambda **kw: pkv.kv_tree_accept([rnd(NB, NKV, BS, D) for _ in range(2)], **a, **kw)


CALLS = (tree, latent, append, accept)


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_every_tensor_is_checked(call):
    args, run = call()
    run()                                                      # as given, it is taken
    for name, t in args.items():
        for what, bad in wrong(t, "k" if name == "kv" else name):
            if what == "size" and name in ("block_tables", "tree_mask", "path"):
                continue                                       # other valid sizes
            if what == "layout" and name == "q" and call is not append:
                bad = torch.cat([t, t], -1)[..., :t.shape[-1]]
            with pytest.raises((pkv.PkvError, ValueError)):
                call(**{name: bad})[1]()
                pytest.fail(f"{name}: {what} was taken")
    torch.cuda.synchronize()
    run()


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_parameters_are_tensors(call):
    args, _ = call()
    call(**{n: torch.nn.Parameter(t, requires_grad=False) for n, t in args.items()})[1]()
    torch.cuda.synchronize()


def test_caches_of_an_accept_are_checked():
    a, _ = accept()
    good = rnd(NB, NKV, BS, D)
    for bad in ([], [good, good.cpu()], [good, good.half()], [good, rnd(NB, NKV, BS, 2 * D)], [good, rnd(NB, NKV, BS, 2 * D)[..., :D]],
                [good, good[None]], [good[0, 0]], [good, None], [good, rnd(NB, NKV, BS, D), good]):
        with pytest.raises((pkv.PkvError, ValueError, TypeError, AttributeError)):
            pkv.kv_tree_accept(bad, **a)
    for out in (a["context_lens"], a["n_accept"], a["q_start"][1:], a["path"].view(-1)[:B]):
        with pytest.raises(pkv.PkvError):                      # new lengths over an input
            pkv.kv_tree_accept([good], **{**a, "new_lens": out})
    with pytest.raises(pkv.PkvError):
        pkv.kv_tree_accept([good], **{**a, "q_start": None})
    torch.cuda.synchronize()


def test_workspaces_that_are_too_small_or_askew_are_refused():
    for call in (tree, latent):
        a, _ = call()
        for bad in (a["workspace"][:-1], torch.cat([a["workspace"], a["workspace"]])[128:]):
            with pytest.raises(pkv.PkvError):
                call(workspace=bad)[1]()
    torch.cuda.synchronize()


OUT = {"tree": "out", "latent": "out", "append": "q_out", "accept": "new_lens"}


def sure(call):
    """Arguments whose results do not depend on what the call before left."""
    a, _ = call()
    caches = [rnd(NB, NKV, BS, D) for _ in range(2)]

    def run(stream, **kw):
        kw = {n: t for n, t in a.items() if n not in kw} | kw
        kw = {n: t for n, t in kw.items() if t is not None}
        if call is accept:
            return pkv.kv_tree_accept(caches, stream=stream, **kw)
        if call is append:
            return pkv.latent_append(table=pkv.rope_table(64, ROPE), stream=stream, **kw)
        fixed = dict(scale=0.125) if call is tree else dict(scale=0.0625, latent=LAT)
        return (pkv.paged_tree_attn if call is tree else pkv.paged_latent_attn)(stream=stream, **fixed, **kw)

    return a, run


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("what", ["output", "workspace"])
def test_buffers_do_not_take_memory_still_in_use(call, what):
    a, run = sure(call)
    name = OUT[call.__name__] if what == "output" else "workspace"
    if name not in a:
        return
    st, expected = torch.cuda.Stream(), run(None).clone()
    copy, want = freed_under_way(a[name].nbytes)
    out = run(st, **{name: None})
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and torch.equal(out, expected)


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_buffers_made_for_a_stream_are_not_given_away_early(call):
    a, run = sure(call)
    st, want = torch.cuda.Stream(), run(None).clone()
    mine = {OUT[call.__name__]: None} | ({"workspace": None} if "workspace" in a else {})
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(SLEEP)                               # the call below waits behind it
    out = run(st, **mine)
    grabbed = [torch.full((t.nbytes,), 77, dtype=torch.uint8, device="cuda") for n, t in a.items() if n in mine]
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda._sleep(SLEEP)
    read = out.clone()
    del out
    with torch.cuda.stream(st):
        taken = torch.full_like(want, 3)
    torch.cuda.synchronize()
    assert torch.equal(read, want) and all(bool((x == 77).all()) for x in grabbed) and bool((taken == 3).all())


@pytest.mark.parametrize("call", (tree, latent, append), ids=lambda f: f.__name__)
def test_calls_from_two_threads(call):
    runs = [sure(call)[1] for _ in range(2)]
    want = [r(None).clone() for r in runs]
    torch.cuda.synchronize()
    got, fails = [None, None], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[i] = [runs[i](None).clone() for _ in range(50)]
            s.synchronize()
        except Exception as e:                                 # noqa: BLE001
            fails.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not fails
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


@pytest.mark.parametrize("call", (tree, latent), ids=lambda f: f.__name__)
def test_two_graphs_share_a_workspace(call):
    """Graphs of other inputs and other shapes of the line in one workspace, replayed in turn on one stream."""
    (a0, run0), (a1, run1) = sure(call), sure(call)
    a1["context_lens"] = a1["context_lens"] - 33
    a1["workspace"] = a0["workspace"]
    want = [run0(None).clone(), run1(None).clone()]
    graphs = []
    for run in (run0, run1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(None)
        graphs.append(g)
    for _ in range(20):
        for a, g, w in zip((a0, a1), graphs, want):
            a["out"].fill_(7)
            g.replay()
            assert torch.equal(a["out"], w)


def test_a_thread_may_begin_with_any_call():
    """Attention as a thread's first CUDA call, where no context is current yet."""
    q, kp, vp, bt, ctx = rnd(B, NH, D), rnd(NB, NKV, BS, D), rnd(NB, NKV, BS, D), TABLES.cuda(), ints(B) + 40
    out, ws = rnd(B, NH, D), torch.empty(pkv.decode_workspace_bytes(B, NH, NKV, D, BS), dtype=torch.uint8, device="cuda")
    want, fails = pkv.paged_decode_attn(q, kp, vp, bt, ctx, 0.125).clone(), []

    def work():
        try:
            pkv.paged_decode_attn(q, kp, vp, bt, ctx, 0.125, out=out, workspace=ws)
        except Exception as e:                                 # noqa: BLE001
            fails.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not fails and torch.equal(out, want)
