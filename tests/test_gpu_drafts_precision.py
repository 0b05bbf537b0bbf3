"""bf16 outputs carry softmax weights of at least 16 bits whatever the batch: a sequence's precision does not depend on which others
share the call, and meets the library's bar for bf16 outputs."""
import pytest
import torch

from drafts_common import check, reference
from gpu_common import BAR_BF16_RELL2, f64, rel_l2
from test_gpu_drafts import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,n_h,ns", [((2, 128), 16, [64, 40, 4, 64]), ((1, 64), 8, [64, 64, 3, 50]), ((512, 64), 128, [1, 1, 1, 1]),
                                         ((512, 64), 32, [8, 2, 5, 8]), ((256, 64), 128, [2, 1, 3, 2]), ((2, 128), 128, [2, 1, 1, 5])])
def test_many_query_rows(kind, n_h, ns):
    for ctx in ([700, 1500, 2500, 64], [6000, 130, 900, 70]):
        c = Case(kind, n_h, 16, [x + n for x, n in zip(ctx, ns)], ns, seed=n_h)
        out, ref = c.run(torch.bfloat16), reference(c)
        check(out, ref, f"{kind} {ns} {ctx}")
        assert rel_l2(f64(out), ref[0]) <= BAR_BF16_RELL2

