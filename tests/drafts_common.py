"""A 64-bit reference of the attention of drafted tokens in torch, for cases too large for the oracle's loops, and the bound
of the kernels' errors (not a test module)."""
import numpy as np
import torch

from gpu_common import DEV, f64


def reference(c, bt=None):
    """(out [T][n_h][v], sum p |v| of the same shape, [T][n_h][1] bound of a score's error) of test_gpu_drafts.Case c in float64.
    Rows of blocks with an id out of range count for nothing; rows of tokens in no sequence are NaN."""
    bt = c.bt if bt is None else bt
    T, n_h, _ = c.q.shape
    pools = [p.to(DEV) for p in c.pools]
    out = torch.full((T, n_h, c.v), float("nan"), dtype=torch.float64, device=DEV)
    size, off = torch.zeros_like(out), torch.zeros(T, n_h, 1, dtype=torch.float64, device=DEV)
    for s, L in enumerate(int(x) for x in c.ctx):
        a, b = int(c.start[s]), int(c.start[s + 1])
        n = b - a
        if n == 0:
            continue
        out[a:b] = 0.0
        if L <= 0:
            continue
        ids = torch.as_tensor(bt[s, :-(-L // c.bs)].astype(np.int64), device=DEV)
        held = (ids >= 0) & (ids < c.blocks)
        held = held.repeat_interleave(c.bs)[:L]
        rows = lambda p: p[ids.clamp(0, c.blocks - 1)].transpose(0, 1).flatten(1, 2)[:, :L].double()  # noqa: E731
        K = rows(pools[0])
        V = K[..., :c.v] if c.latent else rows(pools[1])
        see = torch.ones(n, L, dtype=torch.bool, device=DEV)
        t = torch.arange(L, device=DEV)
        j = t - (L - n)                                        # number among the drafted tokens
        if c.mask is None:
            see &= j[None] <= torch.arange(n, device=DEV)[:, None]
        else:
            words = torch.as_tensor(c.mask[a:b], device=DEV)
            w = (j.clamp(min=0) >> 6)
            bit = (words[:, w.clamp(max=words.shape[1] - 1)] >> (j.clamp(min=0) & 63)) & 1
            see &= (j < 0) | ((bit == 1) & (w < words.shape[1]))
        see &= held
        G = n_h // K.shape[0]
        any_row = see.any(0)
        for g in range(K.shape[0]):
            k, v = K[g].clone(), V[g].clone()
            k[~any_row], v[~any_row] = 0.0, 0.0                # what nobody attends to may be anything
            q = c.q[a:b, g * G:(g + 1) * G].to(DEV).double()
            x = torch.einsum("ihw,tw->iht", q, k) * c.scale
            x = torch.where(see[:, None], x, -torch.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
            total = p.sum(-1, keepdim=True)
            p = p / torch.where(total == 0, 1.0, total)
            out[a:b, g * G:(g + 1) * G] = torch.einsum("iht,tv->ihv", p, v)
            size[a:b, g * G:(g + 1) * G] = torch.einsum("iht,tv->ihv", p, v.abs())
            mag = torch.einsum("ihw,tw->iht", q.abs(), k.abs()).masked_fill(torch.isinf(x), 0.0)
            off[a:b, g * G:(g + 1) * G] = (c.w * 2.0 ** -23 * abs(c.scale)) * mag.amax(-1, keepdim=True)
    return tuple(x.cpu().numpy() for x in (out, size, off))


def check(out, ref, what):
    """A score is an fp32 sum of w products, off by at most w 2^-23 (a step per sum) of the sum of their sizes, `off`; a weight by
    that, and so is their sum: 2 off.  p in two bf16 parts is off by 2^-16 (in three by less), fp32 sums of up to 2^14
    rows of random signs and a rescale per tile by 2^-16; a bf16 output is rounded once, 2^-8 of it."""
    got, (want, size, off) = f64(out), ref
    here = ~np.isnan(want)
    assert np.isfinite(got[here]).all(), (what, "not finite")
    tol = (2 * off + 2.0 ** -15) * size + 1e-6 + (2.0 ** -8 * np.abs(want) if out.dtype == torch.bfloat16 else 0.0)
    worst = (np.abs(got - want) / tol)[here]
    assert worst.max() <= 1.0, (what, str(out.dtype), float(worst.max()), int((worst > 1).sum()))
