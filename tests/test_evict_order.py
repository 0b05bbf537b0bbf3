"""The manager decides before rows move: which sequences are cut, and that nothing of the others changes.  No GPU."""
import pytest

import paged_kv_cache_175_gb300 as pkv


def manager():
    bm = pkv.BlockManager(32, 4)
    prefix = list(range(16))
    bm.add_sequence(1, prefix + [100, 101])                     # 18 tokens
    _, reused = bm.add_sequence(2, prefix + [200, 201, 202])    # shares the first four blocks
    assert reused == 16
    bm.add_sequence(3, [7] * 23)                                # alone
    bm.add_sequence(4, [8] * 6)                                 # short
    return bm


def test_cut_to_leaves_whole_what_may_not_move():
    bm = manager()
    before, lens = bm.tables([1, 2, 3, 4], 8)
    assert bm.cut_to([1, 2, 3, 4], lens, 9) == [18, 19, 9, 6]
    after, now = bm.tables([1, 2, 3, 4], 8)
    assert now.tolist() == [18, 19, 9, 6]
    assert (after[[0, 1, 3]] == before[[0, 1, 3]]).all()
    assert (after[2, :3] == before[2, :3]).all() and (after[2, 3:] == -1).all()
    assert bm.counts()["free"] == 32 - 4 - 1 - 1 - 3 - 2        # shared, the rest of 1 and 2, of 3, and 4
    bm.release(2)
    assert bm.cut_to([1], [18], 9) == [9]                       # alone now
    assert bm.add_sequence(5, list(range(16)) + [1])[1] == 0    # its rows no longer hold the prompt in order


def test_cut_to_a_budget_inside_the_rows_that_are_not_shared_is_refused_too():
    bm = manager()
    assert bm.cut_to([1, 2], [18, 19], 17) == [18, 19]


def test_cut_to_after_a_window_slid():
    bm = manager()
    bm.slide_window(3, 5)
    assert bm.cut_to([3], [23], 9) == [23]


@pytest.mark.parametrize("ids,lens,budget", [([1, 1], [18, 18], 9), ([1], [18, 19], 9), ([3], [23], 0), ([3], [23], -4)])
def test_cut_to_refusals(ids, lens, budget):
    bm = manager()
    with pytest.raises(pkv.PkvError):
        bm.cut_to(ids, lens, budget)
    assert bm.tables([1, 2, 3, 4], 8)[1].tolist() == [18, 19, 23, 6]


def test_every_sequence_between_is_cut_alone():
    bm = manager()
    with pytest.raises(pkv.PkvError):
        bm.evict(1, 9)
    with pytest.raises(pkv.PkvError):
        bm.evict(2, 9)
    assert bm.tables([1, 2], 8)[1].tolist() == [18, 19]
