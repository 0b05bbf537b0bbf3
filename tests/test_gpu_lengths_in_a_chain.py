"""Lengths that change within a chain of the library's own kernels, each launched ahead of the end of the one before, with no
other kernel between: attention, eviction, attention, eviction, attention on one tensor of lengths.  Captured and free runs give the
bits of a run that waits for the device after every call."""
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("op", ["bf16", "mass", "bf16 and mass"])
@pytest.mark.parametrize("B,n_h,n_kv,d,bs,n", [(1, 8, 2, 64, 16, 900), (64, 32, 8, 128, 16, 600), (200, 4, 2, 64, 32, 300)])
def test_attention_behind_an_eviction_sees_its_lengths(op, B, n_h, n_kv, d, bs, n):
    mb = -(-n // bs)
    g = torch.Generator(device=DEV).manual_seed(B)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    q, kp0, vp0, m0 = rnd(B, n_h, d), rnd(B * mb, n_kv, bs, d), rnd(B * mb, n_kv, bs, d), torch.rand(B, n_kv, mb * bs, generator=g, device=DEV)
    bt = torch.randperm(B * mb, generator=g, device=DEV).to(torch.int32).view(B, mb)
    lens0 = (n - torch.arange(B, device=DEV) % 50).to(torch.int32)
    budgets = [(lens0 - 3 - torch.arange(B, device=DEV) % 7).to(torch.int32), lens0 // 2, lens0 // 5]
    kp, vp, lens, st = kp0.clone(), vp0.clone(), [lens0.clone(), lens0.clone()], pkv.alloc_evict_state(B, n_kv, mb * bs, DEV)
    outs = [torch.empty(len(budgets) + 1, B, n_h, d, dtype=torch.bfloat16, device=DEV) for _ in op.split(" and ")]
    ws = {"bf16": torch.empty(pkv.decode_workspace_bytes(B, n_h, n_kv, d, bs), dtype=torch.uint8, device=DEV),
          "mass": torch.empty(pkv.mass_workspace_bytes(B, n_h, n_kv, d, bs, mb), dtype=torch.uint8, device=DEV)}
    we, err = torch.empty(pkv.evict_workspace_bytes(B, n_kv, bs, mb), dtype=torch.uint8, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)

    def attend(i, ctx, wait):
        for o, out in zip(op.split(" and "), outs):
            if o == "bf16":
                pkv.paged_decode_attn(q, kp, vp, bt, ctx, 0.125, out=out[i], workspace=ws[o], err=err)
            else:
                pkv.paged_decode_attn_mass(q, kp, vp, bt, ctx, 0.125, st.mass, out=out[i], workspace=ws[o], err=err)
            wait()

    def chain(wait):
        # the lengths alternate between two tensors (an eviction does not write the one it reads)
        for i, keep in enumerate(budgets):
            attend(i, lens[i % 2], wait)
            pkv.kv_evict(kp, vp, bt, lens[i % 2], keep, 9, st, new_lens=lens[1 - i % 2], workspace=we, err=err)
            wait()
        attend(len(budgets), lens[len(budgets) % 2], wait)

    def reset():
        kp.copy_(kp0), vp.copy_(vp0), st.mass.copy_(m0), st.kept.zero_(), st.dropped.zero_(), st.positions.zero_()
        for x in lens:
            x.copy_(lens0)
        torch.cuda.synchronize()

    def state():
        torch.cuda.synchronize()
        return [x.clone() for x in (*outs, kp, vp, *lens, st.mass, st.positions, st.kept, st.dropped)]

    reset()
    chain(torch.cuda.synchronize)
    want = state()
    assert want[-5 - 1].tolist() != lens0.tolist() and torch.isfinite(want[0].float()).all()
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(lambda: None)
    for k in range(20):
        reset()
        if k % 2:
            graph.replay()
        else:
            chain(lambda: None)
        for i, (a, b) in enumerate(zip(want, state())):
            assert torch.equal(a, b), (k, i)
    assert int(err.item()) == 0
