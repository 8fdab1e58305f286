"""A fork that would take a page from a free list's entry outside the pool changes nothing; entries that it does not
take are not looked at."""
import numpy as np
import pytest

import tensor_transformer_layer_cube_gb300 as t
from oracle import pages as OG
from tests.test_gpu_pages import Book, book

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


@pytest.mark.parametrize("forks", [1, 4, 700])
@pytest.mark.parametrize("entry", ["first", "last"])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, "pages"])
def test_fork_onto_a_page_outside_the_pool(ctx, forks, entry, bad):
    b = book(np.random.default_rng(forks), forks + 1, [5] + [0] * forks, spare=forks + 7)
    count = b.host[3]
    b.host[2][count - 1 if entry == "first" else count - forks] = len(b.host[1]) if bad == "pages" else bad
    b = Book(16, *b.host)
    src, dst, length = [0] * forks, list(range(1, forks + 1)), [33 + i % 15 for i in range(forks)]
    assert not OG.fork(16, *b.host, src, dst, length)[4]
    assert b.check_fork(ctx, src, dst, length) == [] and t.tp3d_sync_status(ctx) == 0


def test_entries_that_a_fork_does_not_take(ctx):
    # of four forks two have a partly filled page; the third entry from the top and all above the count are no pages
    b = book(np.random.default_rng(3), 9, [5, 6, 7] + [0] * 6, spare=12)
    b.host[2][b.host[3] - 3] = -1
    b.host[2][b.host[3]:] = 2 ** 31 - 1
    b = Book(16, *b.host)
    assert len(b.check_fork(ctx, [0, 1, 2, 0], [3, 4, 5, 6], [80, 90, 112, 33])) == 2
    assert t.tp3d_sync_status(ctx) == 0
