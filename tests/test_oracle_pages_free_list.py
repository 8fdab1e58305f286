"""The oracle's fork on a free list with an entry outside the pool."""
import numpy as np
import pytest

from oracle import pages as OG


@pytest.mark.parametrize("bad", [-1, 10, 2 ** 31 - 1, -2 ** 31])
def test_fork_onto_a_page_outside_the_pool_changes_nothing(bad):
    table = [[4, 2, 7], [-1] * 3, [-1] * 3]
    for at in (2, 3):  # the second page taken, the first
        free = [0, 1, 3, 6]
        free[at] = bad
        got, shares, left, copies, fits = OG.fork(16, table, np.zeros(10), free, 4, [0, 0], [1, 2], [17, 40])
        assert not fits and copies == [] and left == 4 and got.tolist() == table and not shares.any()
    # entries that are not taken are not looked at
    assert OG.fork(16, table, np.zeros(10), [0, bad, 3, 6], 4, [0, 0], [1, 2], [17, 40])[3:] == ([(2, 6), (7, 3)], True)
