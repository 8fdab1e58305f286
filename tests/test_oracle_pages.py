"""The oracle of the page operators on cases done by hand, and their refusals,
which come before any launch (so without a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from oracle import pages as OG

EINVAL, ESHAPE, EALIGN, EDTYPE, EUNSUP, EOVER = 1, 2, 3, 4, 7, 8


def test_fork_by_hand():
    table = [[4, 2, 7, -1], [-1] * 4, [9, -1, 5, -1], [-1] * 4, [8] * 4]
    got, shares, left, copies, fits = OG.fork(16, table, np.zeros(10), [0, 1, 3, 6], 4, [0, 2, 0], [1, 3, 4], [40, 48, 32])
    assert fits and left == 3 and copies == [(7, 6)]
    assert got.tolist() == [[4, 2, 7, -1], [4, 2, 6, -1], [9, -1, 5, -1], [9, -1, 5, -1], [4, 2, 8, 8]]
    assert shares.tolist() == [0, 0, 2, 0, 2, 1, 0, 0, 0, 1]
    for src, dst, n in (([0, 0], [1, 1], [16, 16]), ([0, 1], [1, 3], [16, 0]), ([5], [1], [1]), ([0], [-1], [1]),
                        ([0], [1], [65]), ([1], [3], [1]), ([0] * 5, [1, 2, 3, 4, 0], [1] * 5)):
        assert OG.fork(16, table, np.zeros(10), [0, 1, 3, 6], 4, src, dst, n)[3:] == ([], False)


def test_give_back_by_hand():
    table = [[4, 2, 7], [4, 2, 6], [1, -1, 3]]
    got, shares, free, left, fits = OG.give_back(table, [0, 0, 1, 0, 1, 0, 0, 0], [5, -9, -9, -9, -9, -9, -9, -9], 1,
                                                 [0, 1, 0], [3, 3, 2])
    assert fits and got.tolist() == [[-1, -1, -1], [4, -1, -1], [-1, -1, 3]]
    assert free.tolist() == [5, 7, 6, 2, 1, -9, -9, -9] and left == 5 and shares.tolist() == [0, 0, 0, 0, 0, 0, 0, 0]
    assert not OG.give_back([[2, 2]], [0] * 3, [0] * 3, 0, [0], [2])[4]


def test_compact_by_hand():
    got, shares, free, where, copies, fits = OG.compact(16, [[6, 1, 7], [6, 0, -1]], [0, 0, 0, 0, 0, 0, 1, 0],
                                                        [3, 5, 2, 4, 99], 4, [48, 32])
    assert fits and copies == [(6, 2), (7, 3)] and got.tolist() == [[2, 1, 3], [2, 0, -1]]
    assert free.tolist() == [7, 6, 5, 4, 99] and where.tolist() == [0, 1, -1, -1, -1, -1, 2, 3]
    assert shares.tolist() == [0, 0, 1, 0, 0, 0, 0, 0]


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module", autouse=True)
def built():
    t.build()


class Fake:
    """A context's memory of zeros: the checks come before anything in it is used."""

    def __init__(self):
        self.mem = (ctypes.c_char * 4096)()
        self.at = ctypes.addressof(self.mem)


def setting():
    buf = torch.zeros(4096, dtype=torch.int32)
    p = [buf.data_ptr() + 512 * i for i in range(16)]
    return Fake(), buf, p, t.tp3d_page_pool(16, 4, 8, 3, 8, p[0], p[1], p[2])


def check_pool(call):
    """``call(pool, ctx)`` refuses what no pool can be."""
    fake, buf, p, good = setting()

    def pool(**kw):
        x = t.tp3d_page_pool.from_buffer_copy(good)
        for k, v in kw.items():
            setattr(x, k, v)
        return x
    assert call(pool(), None) == EINVAL
    for kw in (dict(rows=-1), dict(pages=0), dict(table_width=-1), dict(free_cap=-1), dict(shares=None),
               dict(free_pages=None), dict(block_table=None)):
        assert call(pool(**kw), fake.at) == EINVAL, kw
    for kw in (dict(page=8), dict(page=24), dict(page=8192), dict(rows=16385), dict(table_width=2 ** 31),
               dict(free_cap=2 ** 31), dict(pages=2 ** 31, free_cap=2 ** 31)):
        assert call(pool(**kw), fake.at) == EUNSUP, kw
    assert call(pool(free_cap=7), fake.at) == ESHAPE
    for k in ("block_table", "shares", "free_pages"):
        assert call(pool(**{k: p[9] + 2}), fake.at) == EALIGN
    assert call(pool(shares=p[0] + 4), fake.at) == EOVER and call(pool(free_pages=p[1] + 8), fake.at) == EOVER


def check_words(call, names, p, overlapping):
    for n in names:
        assert call(**{n: None}) == EINVAL, n
        assert call(**{n: p[10] + 1}) == EALIGN, n
    for a, b in overlapping:
        assert call(**{a: b}) == EOVER, (a, b)


def test_refusals_of_fork():
    fake, buf, p, good = setting()
    lib, names = t.lib(), ("src", "dst", "len", "free_count", "free_left", "copy_from", "copy_to", "copy_count")

    def call(pool=good, ctx=fake.at, forks=2, **kw):
        a = dict(zip(names, p[3:11])) | kw
        return lib.tp3d_paged_fork(ctx, ctypes.byref(pool), forks, *a.values(), None)
    check_pool(lambda pool, ctx: call(pool, ctx))
    check_words(call, names, p, [("src", p[0]), ("free_left", p[6]), ("copy_to", p[8] + 4), ("copy_to", p[10]),
                                 ("copy_count", p[1]), ("copy_from", p[2]), ("dst", p[1] + 8)])
    assert call(forks=-1) == EINVAL and call(forks=16385) == EUNSUP


def test_refusals_of_free():
    fake, buf, p, good = setting()
    lib, names = t.lib(), ("first", "end", "free_count", "free_left")

    def call(pool=good, ctx=fake.at, **kw):
        a = dict(zip(names, p[3:7])) | kw
        return lib.tp3d_paged_free(ctx, ctypes.byref(pool), *a.values(), None)
    check_pool(lambda pool, ctx: call(pool, ctx))
    check_words(call, names, p, [("first", p[0]), ("end", p[2]), ("free_left", p[5]), ("free_count", p[1])])


def test_refusals_of_compact():
    fake, buf, p, good = setting()
    lib, names = t.lib(), ("kv_len", "free_count", "page_map", "copy_from", "copy_to", "copy_count")

    def call(pool=good, ctx=fake.at, **kw):
        a = dict(zip(names, p[3:9])) | kw
        return lib.tp3d_paged_compact(ctx, ctypes.byref(pool), *a.values(), None)
    check_pool(lambda pool, ctx: call(pool, ctx))
    check_words(call, names, p, [("kv_len", p[0]), ("page_map", p[1]), ("copy_from", p[7] + 4), ("copy_count", p[5]),
                                 ("free_count", p[2])])


def test_refusals_of_copy():
    fake, buf, p, _ = setting()
    k, v = (torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16) for _ in range(2))
    lib = t.lib()

    def call(ctx=fake.at, n=2, at=p[0], to=p[1], count=p[2], **kw):
        c = t.kv_cache(k, v)
        for name, x in kw.items():
            setattr(c, name, x)
        return lib.tp3d_paged_copy(ctx, ctypes.byref(c), n, at, to, count, None)
    assert call(n=0) == 0 and call(n=0, at=None, to=None, count=None) == 0
    assert call(ctx=None) == EINVAL and call(n=-1) == EINVAL and call(at=None) == EINVAL and call(to=None) == EINVAL
    assert call(n=2 ** 31) == EUNSUP and call(at=p[0] + 2) == EALIGN and call(count=p[2] + 1) == EALIGN
    assert call(at=k.data_ptr()) == EOVER and call(to=v.data_ptr() + 64) == EOVER and call(count=v.data_ptr()) == EOVER
    assert call(k=None) == EINVAL and call(dtype=0) == EDTYPE and call(page=17) == EUNSUP and call(head_dim=96) == EUNSUP
    assert call(token_stride=0) == EINVAL and call(head_stride=4) == EALIGN


def test_the_bindings_own_checks():
    i32 = dict(dtype=torch.int32)
    table, shares, free, one = torch.zeros(4, 3, **i32), torch.zeros(8, **i32), torch.zeros(8, **i32), torch.zeros(1, **i32)
    pool = t.page_pool(16, table, shares, free)
    assert (pool.rows, pool.pages, pool.table_width, pool.free_cap) == (4, 8, 3, 8)
    for bad in ((table.long(), shares, free), (table, shares.float(), free), (table.t(), shares, free),
                (table[0], shares, free), (table, table, free), (table, shares, free[::2])):
        with pytest.raises(ValueError):
            t.page_pool(16, *bad)
    four, three = torch.zeros(4, **i32), torch.zeros(3, **i32)
    for call in (lambda: t.tp3d_paged_free(None, pool, three, four, one, one, stream=0),
                 lambda: t.tp3d_paged_free(None, pool, four, four.long(), one, one, stream=0),
                 lambda: t.tp3d_paged_fork(None, pool, four, four, three, one, one, four, four, one, stream=0),
                 lambda: t.tp3d_paged_fork(None, pool, four, four, four, one, one, four, three, one, stream=0),
                 lambda: t.tp3d_paged_compact(None, pool, four, one, four, four, four, one, stream=0),
                 lambda: t.tp3d_paged_compact(None, pool, four, one, shares, three, four, one, stream=0),
                 lambda: t.tp3d_paged_copy(None, None, 4, three, four, one, stream=0)):
        with pytest.raises(ValueError):
            call()
