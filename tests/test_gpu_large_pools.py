"""Pools of a hundred thousand pages and more whose low pages are taken (needs an
MI355X): the search for free ones goes over many rounds, and finds the lowest."""
import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
from test_gpu_pages import both, same
from test_gpu_tree import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [100003, 16384 * 9])
def test_free_pages_behind_a_long_row(pages):
    """All but a few pages at the end are taken; a few come back in the middle."""
    rows, page, long = 8, 4, pages - 40
    pool, state = both(pages, rows, long + 10, page)
    for lens in ([long * page] + [0] * 7,
                 [long * page, 40, 9, 0, 1, 0, 0, 0],             # from the end
                 [long * page - 17, 40, 9, 8, 1, 4, 0, 0],        # from what the long row gave back
                 [long * page - 17, 0, 9, 80, 100, 4, 0, 0],      # more than there are
                 [long * page + 100, 40, 9, 80, 9, 4, 0, 0]):
        assert dspark.dspark_resize_pages(*state, i32(lens), page).tolist() == pool.resize(lens)
        same(pool, state)
    at = [long * page - 30, 5, 9, 2, 9, 4, 0, 0]
    src, dst = [2, 2, 4], [5, 6, 7]
    got = dspark.dspark_fork_pages(*state, i32(src), i32(dst), i32(at), page)
    assert list(zip(*[x.tolist() for x in got])) == pool.fork(src, dst, at)
    same(pool, state)


def test_a_pool_that_other_tables_fill():
    """References that this table does not hold: free pages are few and far apart."""
    pages, rows, page = 1 << 20, 30, 16
    free = [5, 16383, 16384, 300000, 300001, 524288, 1000000, (1 << 20) - 2, (1 << 20) - 1]
    pool, state = both(pages, rows, 4, page)
    pool.refs = [1] * pages
    for p in free:
        pool.refs[p] = 0
    state[2].copy_(torch.tensor(pool.refs, dtype=torch.int32))
    for lens in ([16] + [0] * 29, [16, 40, 16] + [0] * 27, [16, 33, 16, 64] + [1] * 26,
                 [0, 33, 16, 48] + [0] * 26, [1] * 9 + [0] * 21):
        assert dspark.dspark_resize_pages(*state, i32(lens), page).tolist() == pool.resize(lens)
        same(pool, state)
