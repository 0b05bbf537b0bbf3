"""Calls on a stream of their own: the buffers they make (outputs, workspaces) never take memory that work queued on the
current stream still uses, nor give theirs to such work too early."""
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, NH, NKV, D, BS, MB = 64, 8, 2, 64, 16, 8
NB = B * MB
SLEEP = 60_000_000                                             # clock cycles: about 30 ms of the current stream


def rnd(*s):
    return torch.randn(*s, device=DEV).to(torch.bfloat16)


class Calls:
    def __init__(self):
        self.q, self.k, self.v, self.kp, self.vp = rnd(B, NH, D), rnd(B, NKV, D), rnd(B, NKV, D), rnd(NB, NKV, BS, D), rnd(NB, NKV, BS, D)
        self.bt = torch.arange(NB, dtype=torch.int32, device=DEV).view(B, MB)
        self.ctx = torch.full((B,), MB * BS, dtype=torch.int32, device=DEV)
        self.pos, self.slots = torch.arange(B, dtype=torch.int32, device=DEV), torch.arange(B, device=DEV) * MB * BS
        self.table, self.c8 = pkv.rope_table(D), pkv.alloc_q8_cache(NB, NKV, BS, D, B, device=DEV)
        self.c4 = pkv.alloc_int4_cache(NB, NKV, BS, D, B, DEV)
        self.state, self.keep = pkv.alloc_evict_state(B, NKV, MB * BS, DEV), self.ctx // 2
        self.ws = {"q8": pkv.q8_workspace_bytes(B, NH, NKV, D, BS), "mass": pkv.mass_workspace_bytes(B, NH, NKV, D, BS, MB),
                   "evict": pkv.evict_workspace_bytes(B, NKV, BS, MB), "bf16": pkv.decode_workspace_bytes(B, NH, NKV, D, BS),
                   "int4": pkv.decode_workspace_bytes(B, NH, NKV, D, BS, int4=True)}

    def run(self, name, stream, **kw):
        """The call's output."""
        if name == "rope_append":
            return pkv.rope_append(self.q, self.k, self.v, self.pos, self.slots, self.table, self.kp, self.vp, stream=stream, **kw)
        if name == "rope_qk":
            return pkv.rope_qk(self.q, self.k, self.pos, self.table, stream=stream, **kw)[0]
        if name == "q8":
            return pkv.paged_decode_attn_q8(self.q, self.c8, self.bt, self.ctx, 0.125, stream=stream, **kw)
        if name == "mass":
            return pkv.paged_decode_attn_mass(self.q, self.kp, self.vp, self.bt, self.ctx, 0.125, self.state.mass, stream=stream, **kw)
        return pkv.kv_evict(self.kp, self.vp, self.bt, self.ctx, self.keep, 4, self.state, stream=stream, **kw)

    def buffers(self, name):
        """Bytes of the output, and of the workspace where there is one, with their keywords."""
        out = {"evict": ("new_lens", self.ctx)}.get(name, ("q_out" if name.startswith("rope") else "out", self.q))
        return (out[0], out[1].nbytes, lambda: torch.empty_like(out[1])), self.ws.get(name)


def freed_under_way(nbytes):
    """A block of nbytes that is freed while the current stream's queued copy of it has not run; returns (copy, values)."""
    a = torch.randint(0, 256, (nbytes,), dtype=torch.uint8, device=DEV)
    want = a.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    return a.clone(), want                                     # a dies with its copy still in the queue


NEW = ["rope_append", "rope_qk", "q8", "mass", "evict"]


@pytest.mark.parametrize("name", NEW)
def test_outputs_do_not_take_memory_still_in_use(name):
    c, st = Calls(), torch.cuda.Stream()
    (key, nbytes, make), ws = c.buffers(name)
    kw = {} if ws is None else {"workspace": torch.empty(ws, dtype=torch.uint8, device=DEV)}
    c.run(name, None, **kw, **{key: make()})
    copy, want = freed_under_way(nbytes)
    out = c.run(name, st, **kw)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and out.nbytes == nbytes


@pytest.mark.parametrize("name", ["q8", "mass", "evict"])
def test_workspaces_do_not_take_memory_still_in_use(name):
    c, st = Calls(), torch.cuda.Stream()
    (key, _, make), ws = c.buffers(name)
    out = make()
    c.run(name, None, **{key: out})
    copy, want = freed_under_way(ws)
    c.run(name, st, **{key: out})
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


@pytest.mark.parametrize("name", NEW)
def test_buffers_made_for_a_stream_are_not_given_away_early(name):
    # the output freed while the current stream still reads it; the workspace while the side stream's work has not run
    c, st = Calls(), torch.cuda.Stream()
    want = c.run(name, None).clone()
    if name == "evict":
        c.state.kept.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(SLEEP)                               # the call below waits behind it
    out = c.run(name, st)
    grabbed = [torch.full((n,), 77, dtype=torch.uint8, device=DEV) for n in c.ws.values()]   # on the current stream, at once
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda._sleep(SLEEP)
    read = out.clone()
    del out
    with torch.cuda.stream(st):
        taken = torch.full_like(want, 3)
    torch.cuda.synchronize()
    assert torch.equal(read, want) and all(bool((x == 77).all()) for x in grabbed) and bool((taken == 3).all())


class OlderCalls(Calls):
    """The bf16 and INT4 attention, the deviation and the selection."""

    def run(self, name, stream, **kw):
        if name == "bf16":
            return pkv.paged_decode_attn(self.q, self.kp, self.vp, self.bt, self.ctx, 0.125, stream=stream, **kw)
        if name == "noalloc":
            return pkv.paged_decode_attn_noalloc(self.q, self.kp, self.vp, self.bt, self.ctx, 0.125, stream=stream, **kw)
        if name == "int4":
            return pkv.paged_decode_attn_int4(self.q, self.c4, self.bt, self.ctx, 0.125, stream=stream, **kw)
        if name == "deviation":
            return pkv.kv_deviation(self.kp, self.vp, self.slots, self.k, self.v, stream=stream, **kw)
        return pkv.select_top(self.k.float().view(-1), [0, 1000, 5000], [100, 900], stream=stream, **kw)

    def buffers(self, name):
        nbytes = {"deviation": 4 * B, "select": 4 * 1000}.get(name, self.q.nbytes)
        return ("out", nbytes, None), self.ws.get(name)


OLDER = ["bf16", "noalloc", "int4", "deviation", "select"]


@pytest.mark.parametrize("name", OLDER)
def test_older_outputs_do_not_take_memory_still_in_use(name):
    c, st = OlderCalls(), torch.cuda.Stream()
    (_, nbytes, _), ws = c.buffers(name)
    kw = {} if ws is None else {"workspace": torch.empty(ws, dtype=torch.uint8, device=DEV)}
    want_out = c.run(name, None, **kw)
    copy, want = freed_under_way(nbytes)
    out = c.run(name, st, **kw)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and torch.equal(out, want_out) and out.nbytes == nbytes


@pytest.mark.parametrize("name", ["bf16", "int4"])
def test_older_workspaces_do_not_take_memory_still_in_use(name):
    c, st = OlderCalls(), torch.cuda.Stream()
    out = c.run(name, None)
    copy, want = freed_under_way(c.ws[name])
    c.run(name, st, out=out)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
