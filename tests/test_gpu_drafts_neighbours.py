"""A token's output does not depend, to the last bit, on the queries of other sequences or of other kv heads' groups, although
they lie in the same row tile."""
import numpy as np
import pytest
import torch

from test_gpu_drafts import Case

pytestmark = pytest.mark.gpu
CTX = [600, 150, 300]


def case(kind, n_h, ns):
    """Keys whose last channel grows within a tile: queries with a large number there raise a tile's offsets."""
    c = Case(kind, n_h, 16, CTX, ns, seed=n_h, mask=None)
    for s, L in enumerate(CTX):
        t = np.arange(L)
        c.pools[0][c.bt[s, t // 16], :, t % 16, -1] = torch.as_tensor(t // 16 % 8).to(torch.bfloat16)[:, None]
    c.q[..., -1] = 0.0
    return c


@pytest.mark.parametrize("kind,n_h,ns", [((2, 128), 8, [1, 3, 1]), ((1, 64), 5, [2, 4, 1]), ((2, 128), 8, [5, 9, 3]), ((2, 128), 8, [9, 20, 11]),
                                         ((512, 64), 4, [1, 2, 1]), ((512, 64), 8, [3, 4, 2]), ((256, 64), 24, [2, 3, 5]), ((512, 64), 40, [3, 1, 2])])
def test_queries_of_the_next_sequence(kind, n_h, ns):
    c = case(kind, n_h, ns)
    for dtype in (torch.float32, torch.bfloat16):
        c.q[..., -1] = 0.0
        want = c.run(dtype)
        for value in (900.0, -900.0, float("inf"), float("nan")):
            c.q[ns[0]:, :, -1] = value
            assert torch.equal(c.run(dtype)[:ns[0]], want[:ns[0]]), (dtype, value)


@pytest.mark.parametrize("n", [1, 2])
def test_queries_of_the_next_group(n):
    # 40 heads to a group: its second row tile begins with 8 of them, behind which the next group's lie
    c = case((2, 128), 80, [n] * 3)
    for dtype in (torch.float32, torch.bfloat16):
        c.q[..., -1] = 0.0
        want = c.run(dtype)
        for value in (900.0, float("inf")):
            c.q[:, 40:, -1] = value
            assert torch.equal(c.run(dtype)[:, :40], want[:, :40]), (dtype, value)
