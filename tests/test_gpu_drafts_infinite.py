"""Scores of minus infinity (keys that hold it, or finite ones whose product overflows) have weight zero, wherever they lie: at the
start of a sequence, of a tile, of a part of a cut segment, ahead of scores that raise the offsets."""
import numpy as np
import pytest
import torch

from drafts_common import check, reference
from gpu_common import f64
from test_gpu_drafts import Case

pytestmark = pytest.mark.gpu
KINDS = [pytest.param(k, h, n, id=f"{k[0]}_{k[1]}_h{h}_n{n}") for k, h, n in
         [((2, 128), 8, 2), ((2, 128), 8, 6), ((2, 64), 16, 7), ((512, 64), 16, 1), ((512, 64), 16, 2), ((256, 32), 40, 2)]]


def case(kind, n_h, n, ctx, bad, value=-float("inf"), rise=0):
    """The rows that `bad` names have a score of minus infinity for all query rows; with `rise`, every other head's scores grow along the
    context by so much (base 2) every 64 rows."""
    c = Case(kind, n_h, 16, ctx, [min(n, x) for x in ctx], seed=sum(ctx) + n, mask=None)
    k = c.pools[0]
    c.q[..., -1] = 4.0
    c.q[..., -2] = 0.0
    c.q[:, ::2, -2] = rise / (c.scale * 1.4426950408889634)
    for s, L in enumerate(ctx):
        t = np.arange(L)
        blk, row = c.bt[s, t // 16], t % 16
        k[blk, :, row, -1] = 0.0
        k[blk, :, row, -2] = torch.as_tensor(t // 64).to(torch.bfloat16)[:, None]
        b = t[[bool(bad(x)) and x < L - 1 for x in t]]          # a row is left to attend to
        k[c.bt[s, b // 16], :, b % 16, -1] = value
    return c


ROWS = {"first": lambda t: t == 0, "tile_starts": lambda t: t % 64 == 0, "a_tile": lambda t: t < 128, "late_tiles": lambda t: 128 <= t < 384,
        "most": lambda t: t % 5}


@pytest.mark.parametrize("bad", ROWS, ids=str)
@pytest.mark.parametrize("kind,n_h,n", KINDS)
def test_rows_of_minus_infinity(kind, n_h, n, bad):
    for ctx in ([40], [300, 17, 129], [9000], [1500] * 40):
        c = case(kind, n_h, n, ctx, ROWS[bad])
        ref = reference(c)
        for dtype in (torch.float32, torch.bfloat16):
            check(c.run(dtype), ref, f"{ctx[:3]} {bad}")


@pytest.mark.parametrize("bad", ["first", "tile_starts", "a_tile"])
@pytest.mark.parametrize("kind,n_h,n", KINDS)
def test_offsets_raised_behind_them(kind, n_h, n, bad):
    for ctx in ([300, 700], [3000] * 24):
        c = case(kind, n_h, n, ctx, ROWS[bad], rise=40)
        check(c.run(), reference(c), f"{ctx[:3]} {bad}")


@pytest.mark.parametrize("kind,n_h,n", KINDS)
def test_finite_keys_whose_scores_overflow(kind, n_h, n):
    for ctx in ([100], [700, 2000]):
        c = case(kind, n_h, n, ctx, ROWS["tile_starts"], value=-3e38)
        check(c.run(), reference(c), str(ctx))


@pytest.mark.parametrize("kind,n_h,n", KINDS)
def test_nothing_but_minus_infinity(kind, n_h, n):
    # no row that counts: zeros, as where nothing is attended to
    c = case(kind, n_h, n, [150, 40], lambda t: False)
    c.pools[0][..., -1] = -float("inf")
    assert not f64(c.run()).any()
