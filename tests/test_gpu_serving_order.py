"""A decode loop whose lengths, positions and slots are computed on the GPU right before the calls: run
freely, captured into a graph, and with the device waited for after every call, it gives the same bits.
(The kernels start while the one before them ends; what they read early must be there.)"""
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def loop(kind, B, n_h, n_kv, d, bs, ctx0, steps, mode):
    """`steps` decode steps; mode: free, waited or graph.  Returns every step's output and the caches."""
    mb = -(-(ctx0 + steps + 1) // bs)
    nb, T = B * mb, mb * bs
    g = torch.Generator().manual_seed(B + n_h)
    new = torch.randn(steps, B, n_h + 2 * n_kv, d, generator=g).to(torch.bfloat16).to(DEV)
    kp, vp = (torch.randn(nb, n_kv, bs, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    bt = torch.randperm(nb, generator=g).to(torch.int32).reshape(B, mb).to(DEV)
    table = pkv.rope_table(d)
    ctx = (ctx0 - torch.arange(B, dtype=torch.int32) % 7).to(DEV)
    lens = torch.full((B,), ctx0 - 5, dtype=torch.int32, device=DEV)
    seq, rows = torch.arange(B, dtype=torch.int32, device=DEV), torch.arange(B, device=DEV)
    pos, slots, at = torch.zeros_like(ctx), torch.zeros(B, dtype=torch.int64, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    x, err = torch.empty_like(new[0]), torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = torch.zeros(steps, B, n_h, d, dtype=torch.bfloat16, device=DEV)
    q_rot, out = torch.empty(B, n_h, d, dtype=torch.bfloat16, device=DEV), torch.empty(B, n_h, d, dtype=torch.bfloat16, device=DEV)
    cache = pkv.alloc_q8_cache(nb, n_kv, bs, d, B, device=DEV)
    st = pkv.alloc_evict_state(B, n_kv, T, DEV)
    if kind == "q8":
        for b in range(B):                                     # the context so far
            n = int(ctx[b])
            t = torch.arange(n, device=DEV)
            pkv.kv_quant_append_q8(kp.transpose(1, 2).reshape(-1, n_kv, d)[:n], vp.transpose(1, 2).reshape(-1, n_kv, d)[:n],
                                   bt[b].long()[t // bs] * bs + t % bs, seq[b].expand(n).contiguous(), cache, err=err)
        ws = torch.empty(pkv.q8_workspace_bytes(B, n_h, n_kv, d, bs), dtype=torch.uint8, device=DEV)
        k_rot = torch.empty(B, n_kv, d, dtype=torch.bfloat16, device=DEV)
    else:
        ws = torch.empty(pkv.mass_workspace_bytes(B, n_h, n_kv, d, bs, mb), dtype=torch.uint8, device=DEV)
        we = torch.empty(pkv.evict_workspace_bytes(B, n_kv, bs, mb), dtype=torch.uint8, device=DEV)
        new_lens = torch.empty_like(ctx)
    wait = torch.cuda.synchronize if mode == "waited" else (lambda: None)

    def step():
        x.copy_(new.index_select(0, at)[0])
        pos.copy_(st.dropped + ctx)
        slots.copy_(bt[rows, (ctx // bs).long()].long() * bs + ctx % bs)
        ctx.add_(1)
        wait()
        q, k, v = x[:, :n_h], x[:, n_h:n_h + n_kv], x[:, n_h + n_kv:]
        if kind == "q8":
            pkv.rope_qk(q, k, pos, table, q_out=q_rot, k_out=k_rot)
            wait()
            pkv.kv_quant_append_q8(k_rot, v, slots, seq, cache, err=err)
            wait()
            pkv.paged_decode_attn_q8(q_rot, cache, bt, ctx, d ** -0.5, out=out, workspace=ws, err=err)
        else:
            pkv.rope_append(q, k, v, pos, slots, table, kp, vp, q_out=q_rot, err=err)
            wait()
            pkv.paged_decode_attn_mass(q_rot, kp, vp, bt, ctx, d ** -0.5, st.mass, out=out, workspace=ws, err=err)
            wait()
            pkv.kv_evict(kp, vp, bt, ctx, lens, 4, st, new_lens=new_lens, workspace=we, err=err)
            ctx.copy_(new_lens)
        outs.index_copy_(0, at, out[None])
        at.add_(1)
        wait()

    if mode == "graph":
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(steps - 1):
            graph.replay()
    else:
        for _ in range(steps):
            step()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return [outs, ctx] + ([cache.records, cache.k_tail, cache.v_tail] if kind == "q8" else
                          [kp, vp, st.mass, st.positions, st.kept, st.dropped])


@pytest.mark.parametrize("kind", ["q8", "evict"])
@pytest.mark.parametrize("B,n_h,n_kv,d,bs,ctx0", [(3, 8, 2, 64, 16, 40), (64, 32, 8, 128, 16, 90), (300, 4, 1, 64, 32, 37)])
def test_free_waited_and_captured_loops_agree(kind, B, n_h, n_kv, d, bs, ctx0):
    want = loop(kind, B, n_h, n_kv, d, bs, ctx0, 24, "waited")
    assert torch.isfinite(want[0].float()).all()
    for mode in ("free", "graph"):
        got = loop(kind, B, n_h, n_kv, d, bs, ctx0, 24, mode)
        for i, (a, b) in enumerate(zip(want, got)):
            assert torch.equal(a, b), (mode, i)
