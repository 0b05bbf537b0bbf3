"""How many bits of the softmax weights reach the output: accounted and 8-bit attention against the formula in
64 bits, with bounds on the row's own sum of p |v|."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_175_gb300 as pkv
from gpu_common import DEV, err_flag, f64

pytestmark = pytest.mark.gpu


def weights(q, k, scale):
    """p [heads][tokens] of queries [heads][d] over keys [tokens][d], in 64 bits."""
    x = scale * q @ k.T
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_h", [1, 3, 4, 5, 8, 16, 24, 32, 64])
def test_accounted_attention_carries_every_bit_of_the_weights(n_h, d):
    """One kv head whose value rows are unit vectors, so that output channel c is the weight of token c + 1 alone
    (token 0 has the zero row).  A score is one product of bf16 values, exact in fp32.  In base-2 units scores lie in
    [0, 1.81], so a weight is off by: score and offset (scale * log2 e, the product, the difference)
    2^-21 ln 2 = 3.4e-7; two exponentials (its own, the merge's) 2^-22 each; the sum's terms as much again, its
    additions over at most 12 roundings; division and products 6 roundings of 2^-24: 2.5e-6 < 2^-18 in all.  Weights
    cut to 16 bits are off by up to 2^-17."""
    bs, T, scale = 16, d + 1, 0.125
    g = torch.Generator().manual_seed(n_h + d)
    q = torch.zeros(3, n_h, d)
    q[..., 0] = 1 + torch.rand(3, n_h, generator=g)
    k = torch.zeros(T, d)
    k[:, 0] = 5 * torch.rand(T, generator=g)
    v = torch.zeros(T, d)
    v[1:] = torch.eye(d)
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    blocks = -(-T // bs)
    pool = torch.zeros(2, blocks * bs, d, dtype=torch.bfloat16)
    pool[0, :T], pool[1, :T] = k, v
    kp, vp = (x.view(blocks, 1, bs, d).to(DEV) for x in pool)
    bt = torch.arange(blocks, dtype=torch.int32, device=DEV).expand(3, -1).contiguous()
    ctx = torch.full((3,), T, dtype=torch.int32, device=DEV)
    mass, err = torch.zeros(3, 1, blocks * bs, device=DEV), err_flag()
    out = f64(pkv.paged_decode_attn_mass(q.to(DEV), kp, vp, bt, ctx, scale, mass, out_dtype=torch.float32, err=err))
    assert int(err.item()) == 0
    for s in range(3):
        p = weights(f64(q[s]), f64(k), scale)
        assert np.abs(out[s] / p[:, 1:] - 1).max() < 2.0 ** -18
        assert np.abs(f64(mass)[s, 0, :T] / p.sum(0) - 1).max() < 2.0 ** -18


@pytest.mark.parametrize("op", ["mass", "q8"])
@pytest.mark.parametrize("n_h,n_kv", [(4, 1), (5, 1), (16, 2), (16, 1), (32, 1), (64, 1)])
def test_bf16_outputs_are_off_by_the_rows_own_weights(op, n_h, n_kv):
    """|error| <= 2^-8 |out| (the output's rounding) and, of the row's own sum p |v|: the rounding of p (2^-11 fp16 in the
    8-bit attention, 2^-17 a bf16 pair in the accounted one, for larger groups), twice the score's absolute error (fp32
    sums of d products: (d + 8) 2^-24 sum |q k| at most) and 2^-19 for exponentials, sum and division."""
    d, bs, lens = 64, 16, [200, 33, 1, 77]
    g = torch.Generator().manual_seed(n_h)
    nb = [-(-n // bs) for n in lens]
    bt = np.full((len(lens), max(nb)), -1, np.int32)
    for s, n in enumerate(nb):
        bt[s, :n] = sum(nb[:s]) + np.arange(n)
    kp, vp = (torch.randn(sum(nb), n_kv, bs, d, generator=g).to(torch.bfloat16) for _ in range(2))
    vp *= torch.exp2(torch.randint(-10, 10, (sum(nb), 1, 1, 1), generator=g)).to(torch.bfloat16)   # rows far below the largest value
    q = torch.randn(len(lens), n_h, d, generator=g).to(torch.bfloat16)
    dbt, ctx, err = torch.as_tensor(bt, device=DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), err_flag()
    if op == "mass":
        held, of_p = (f64(kp), f64(vp)), (2.0 ** -17 if n_h // n_kv > 8 else 0.0)
        out = pkv.paged_decode_attn_mass(q.to(DEV), kp.to(DEV), vp.to(DEV), dbt, ctx, 0.125, torch.zeros(len(lens), n_kv, bt.shape[1] * bs, device=DEV), err=err)
    else:
        of_p = 2.0 ** -11 if n_h // n_kv > 4 else 0.0
        c = pkv.alloc_q8_cache(sum(nb), n_kv, bs, d, len(lens), "int8", DEV)
        rows = [x.transpose(1, 2).reshape(-1, n_kv, d).to(DEV) for x in (kp, vp)]                  # every block filled
        seq = torch.as_tensor(np.repeat(np.arange(len(lens)), np.array(nb) * bs).astype(np.int32), device=DEV)
        pkv.kv_quant_append_q8(*rows, torch.arange(sum(nb) * bs, device=DEV), seq, c, err=err)
        sc = c.scales.double().cpu().numpy()
        held = tuple(f64(x.float()) * sc[:, :, i, None, None] for i, x in enumerate((c.k_codes, c.v_codes)))
        out = pkv.paged_decode_attn_q8(q.to(DEV), c, dbt, ctx, 0.125, err=err)
    assert int(err.item()) == 0 and out.dtype == torch.bfloat16
    got, G = f64(out), n_h // n_kv
    for s, n in enumerate(lens):
        for h in range(n_kv):
            k, v = (oracle.gather_sequence(x, bt[s], n, h, bs) for x in held)
            qa = f64(q[s, h * G:(h + 1) * G])
            p = weights(qa, k, 0.125)
            delta = 2.0 ** -24 * (d + 8) * 0.125 * (np.abs(qa) @ np.abs(k).T).max(-1, keepdims=True)
            own = (of_p + 2 * delta + 2.0 ** -19) * (p @ np.abs(v))
            ref = p @ v
            assert np.all(np.abs(got[s, h * G:(h + 1) * G] - ref) <= 2.0 ** -8 * np.abs(ref) + own * (1 + 2.0 ** -8)), (s, h)
