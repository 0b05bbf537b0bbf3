"""Inputs written on the GPU by the kernel directly ahead of a call: lengths, positions, slots, budgets.  The calls run
freely, captured into a graph, and with the device waited for in between; all give the same bits."""
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(n, start=0, dtype=torch.int32):
    return torch.arange(start, start + n, dtype=dtype, device=DEV)


def run(step, reset, outs, steps, mode):
    """The outputs after each of `steps` steps; mode: waited (step gets a synchronize to call), free or graph."""
    reset()
    got = []
    nothing = lambda: None  # noqa: E731
    if mode == "graph":
        step(nothing)                                          # sets the kernels up
        torch.cuda.synchronize()
        reset()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(nothing)
        reset()
    for _ in range(steps):
        if mode == "graph":
            g.replay()
        else:
            step(torch.cuda.synchronize if mode == "waited" else nothing)
        got.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    return got


def check(step, reset, outs, steps=30):
    want = run(step, reset, outs, steps, "waited")
    assert not torch.equal(want[0][0], want[-1][0])             # the steps do differ
    for mode in ("free", "graph"):
        for i, (a, b) in enumerate(zip(want, run(step, reset, outs, steps, mode))):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), (mode, i)


@pytest.mark.parametrize("op", ["mass", "q8"])
@pytest.mark.parametrize("B,n_h,n_kv,d,bs,ctx0", [(1, 8, 2, 64, 16, 100), (64, 32, 8, 128, 16, 300), (250, 4, 1, 64, 32, 37), (300, 8, 2, 64, 64, 60)])
def test_lengths_written_by_the_kernel_ahead(op, B, n_h, n_kv, d, bs, ctx0):
    mb = -(-(ctx0 + 200) // bs)
    g = torch.Generator(device=DEV).manual_seed(B)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    bt = torch.randperm(B * mb, generator=g, device=DEV).to(torch.int32).view(B, mb)
    q, out, ctx, err = rnd(B, n_h, d), torch.empty(B, n_h, d, dtype=torch.bfloat16, device=DEV), ints(B), torch.zeros(1, dtype=torch.int32, device=DEV)
    lens0 = ctx0 - ints(B) % 13
    if op == "mass":
        kp, vp, mass = rnd(B * mb, n_kv, bs, d), rnd(B * mb, n_kv, bs, d), torch.zeros(B, n_kv, mb * bs, device=DEV)
        ws = torch.empty(pkv.mass_workspace_bytes(B, n_h, n_kv, d, bs, mb), dtype=torch.uint8, device=DEV)
        call = lambda: pkv.paged_decode_attn_mass(q, kp, vp, bt, ctx, 0.125, mass, out=out, workspace=ws, err=err)  # noqa: E731
    else:
        mass = torch.zeros(1, device=DEV)
        c = pkv.alloc_q8_cache(B * mb, n_kv, bs, d, 1, "int8", DEV)
        c.records[:, :, :2 * bs * d] = torch.randint(0, 256, (B * mb, n_kv, 2 * bs * d), generator=g, device=DEV).to(torch.uint8)
        c.scales.fill_(0.01)
        ws = torch.empty(pkv.q8_workspace_bytes(B, n_h, n_kv, d, bs, "int8"), dtype=torch.uint8, device=DEV)
        call = lambda: pkv.paged_decode_attn_q8(q, c, bt, ctx, 0.125, out=out, workspace=ws, err=err)  # noqa: E731

    def step(wait):
        ctx.add_(5)                                            # nothing lies between this kernel and the call
        wait()
        call()

    def reset():
        ctx.copy_(lens0)
        mass.zero_()

    check(step, reset, [out, mass])
    assert int(err.item()) == 0


def test_positions_slots_and_budgets_written_by_the_kernel_ahead():
    B, n_h, n_kv, d, bs, mb = 16, 8, 2, 64, 16, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    q, k, v, kp0, vp0 = rnd(B, n_h, d), rnd(B, n_kv, d), rnd(B, n_kv, d), rnd(B * mb, n_kv, bs, d), rnd(B * mb, n_kv, bs, d)
    kp, vp, q_out, k_out = kp0.clone(), vp0.clone(), torch.empty_like(q), torch.empty_like(k)
    pos, slots, seq, table = ints(B), ints(B, dtype=torch.int64), ints(B), pkv.rope_table(d)
    c = pkv.alloc_q8_cache(B * mb, n_kv, bs, d, B, device=DEV)

    def step(wait):
        pos.add_(3)
        wait()
        pkv.rope_qk(q, k, pos, table, q_out=q_out, k_out=k_out)
        wait()
        slots.add_(1)
        wait()
        pkv.kv_quant_append_q8(k_out, v, slots, seq, c)
        wait()
        slots.add_(0)
        wait()
        pkv.rope_append(q, k, v, pos, slots, table, kp, vp, q_out=q_out)

    def reset():
        kp.copy_(kp0), vp.copy_(vp0), pos.copy_(ints(B)), slots.copy_(ints(B, dtype=torch.int64) * mb * bs)
        c.records.zero_(), c.k_tail.zero_(), c.v_tail.zero_()

    check(step, reset, [q_out, k_out, kp, vp, c.records, c.k_tail, c.v_tail], 40)

    bt, ctx, keep, new = ints(B * mb).view(B, mb), ints(B), ints(B), ints(B)
    st = pkv.alloc_evict_state(B, n_kv, mb * bs, DEV)
    m0 = torch.rand(B, n_kv, mb * bs, generator=g, device=DEV)
    ws = torch.empty(pkv.evict_workspace_bytes(B, n_kv, bs, mb), dtype=torch.uint8, device=DEV)

    def evict(wait):
        keep.sub_(7)
        wait()
        pkv.kv_evict(kp, vp, bt, ctx, keep, 5, st, new_lens=new, workspace=ws)
        wait()
        ctx.copy_(new)

    def reset_evict():
        kp.copy_(kp0), vp.copy_(vp0), keep.fill_(mb * bs), ctx.fill_(mb * bs)
        st.mass.copy_(m0), st.kept.zero_(), st.dropped.zero_(), st.positions.zero_()

    check(evict, reset_evict, [new, kp, vp, st.mass, st.positions, st.kept, st.dropped], 20)
