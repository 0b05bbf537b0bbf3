"""Eviction of more rows than a cluster's registers hold (over 131072): equal accounts at the cut, recorded positions, several
heads and sequences, in place and to another state, K and V apart; all against the oracle."""
import numpy as np
import pytest

from test_gpu_evict import check_evict, pools, pytestmark, state_of  # noqa: F401


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("ties", [True, False])
@pytest.mark.parametrize("lens,keep,recent,kept", [([131073 + 64], [40000], 1000, [100000]),
                                                   ([140001, 3, 9000, 140000], [139000, 1, 9000, 7], 50, [0, 3, 4000, 139999]),
                                                   ([133000], [0], 5, [1]), ([133000, 132000], [65000, 131999], 0, [66000, 500])])
def test_many_rows(lens, keep, recent, kept, ties, in_place):
    bs, n_kv = 64, 2
    kp, vp, bt, _ = pools(lens, n_kv, 64, bs, seed=len(lens))
    T = bt.shape[1] * bs
    assert T > 131072
    st = state_of(len(lens), n_kv, T, lens, kept, np.random.default_rng(keep[0]), ties)
    if ties:                                                   # the cut falls among rows of one account
        for s, n in enumerate(lens):
            cut = np.sort(st[0][s, 0, :n])[::-1][min(keep[s], n - 1)]
            assert min(n, keep[s]) < 1000 or np.count_nonzero(st[0][s, 0, :n] == cut) > 1
    check_evict(kp, vp, bt, lens, keep, recent, st, bs, in_place)
