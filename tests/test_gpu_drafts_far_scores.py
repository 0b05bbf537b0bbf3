"""Scores whose size leaves no bits for their differences' fractions: the largest one's weight is 1 all the same, wherever it lies."""
import numpy as np
import pytest
import torch

from drafts_common import reference
from gpu_common import f64
from test_gpu_drafts import Case

pytestmark = pytest.mark.gpu
KINDS = [pytest.param(k, h, n, id=f"{k[0]}_{k[1]}_h{h}_n{n}") for k, h, n in
         [((2, 128), 8, 2), ((2, 128), 8, 6), ((2, 64), 40, 7), ((512, 64), 16, 1), ((512, 64), 16, 2), ((256, 32), 40, 2)]]


def case(kind, n_h, n, ctx):
    c = Case(kind, n_h, 16, ctx, [min(n, x) for x in ctx], seed=sum(ctx) + n, mask=None)
    c.q[:] = 0.0
    c.q[..., -1] = 1.0
    return c


@pytest.mark.parametrize("size", [1e38, 3e30, 1e12, 4e7])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("kind,n_h,n", KINDS)
def test_equal_scores_far_from_zero(kind, n_h, n, sign, size):
    # the average of the values, with an offset of any size
    for ctx in ([1], [40, 200], [5000], [700] * 30):
        c = case(kind, n_h, n, ctx)
        c.pools[0][..., -1] = sign * size
        want, mag, _ = reference(c)
        for dtype in (torch.float32, torch.bfloat16):
            got = f64(c.run(dtype))
            # equal weights: fp32 sums of up to 2^13 rows of random signs, and the output's own rounding
            assert (np.abs(got - want) <= 2.0 ** -16 * mag + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0) + 1e-7).all(), ctx


@pytest.mark.parametrize("kind,n_h,n", KINDS)
def test_one_of_them_far_above_the_others(kind, n_h, n):
    # whole powers of two as scores (before the scale): the largest takes all, behind others that were the largest before
    for at in ([0], [130], [0, 70, 130, 260, 399], [399]):
        c = case(kind, n_h, n, [400 + n, 390])
        k = c.pools[0]
        k[..., -1] = -1e37
        for i, t in enumerate(at):
            k[c.bt[0, t // 16], :, t % 16, -1] = 2.0 ** (20 + 15 * i)
        want = reference(c)[0]
        for dtype in (torch.float32, torch.bfloat16):
            got = f64(c.run(dtype))
            a = int(c.start[1])
            assert np.array_equal(got[:a], want[:a]), (at, dtype)            # that row's values, which bf16 holds
            assert np.isfinite(got).all()
