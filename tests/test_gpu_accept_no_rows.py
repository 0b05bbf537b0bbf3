"""kv_tree_accept of sequences without cached rows: drafted tokens that nothing holds, and counts out of range, are flagged; a
padded sequence, of which nothing is accepted, is not."""
import pytest
import torch

import paged_kv_cache_175_gb300 as pkv
from gpu_common import DEV, err_flag

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [0, 6])
@pytest.mark.parametrize("count", [0, 2, 9, -1])
def test_no_rows(n, count):
    to = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pool = torch.randn(4, 2, 16, 64, device=DEV).bfloat16()
    before, err = pool.clone(), err_flag()
    lens = pkv.kv_tree_accept([pool], to([0, 1], [2, 3]), to(0, 20), to(0, n, n + 3), to([0, 1, 3], [0, 1, 2]), to(count, 3), err=err)
    assert lens.tolist() == [0, 20] and torch.equal(pool, before)
    assert int(err.item()) == (pkv.DEV_BAD_TREE if count else 0)
