"""Pages that rows of a block table get, give back and share, against lists on the
CPU (needs an MI355X), and copies of pages."""
import random

import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
import tree_ref as ref
from test_gpu_tree import i32, on_device, pools, same_bytes

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def same(pool, state):
    table, held, refs = state
    assert held.tolist() == pool.held
    assert refs.tolist() == pool.refs
    assert table.tolist() == pool.table


def both(pages, rows, width, page):
    return ref.Pool(pages, rows, width, page), dspark.page_pool(pages, rows, width, DEV)


@pytest.mark.parametrize("pages,rows,width,page", [
    (1, 1, 1, 1), (100, 5, 30, 16), (40, 9, 12, 7), (5000, 300, 40, 64), (3000, 1500, 8, 16),
    (40000, 3, 20000, 16)])
def test_resize(pages, rows, width, page):
    pool, state = both(pages, rows, width, page)
    for turn in range(6):
        hi = width * page * (2 if turn == 3 else 1) // (1 if turn % 2 else 3)
        lens = ref.some_lens(turn + rows, rows, max(hi, 1))
        if turn == 4:
            lens[0] = -5
        granted = dspark.dspark_resize_pages(*state, i32(lens), page)
        assert granted.tolist() == pool.resize(lens)
        same(pool, state)
    dspark.dspark_resize_pages(*state, i32([0] * rows), page)
    assert int(state[2].abs().sum()) == 0 and bool((state[0] == -1).all())


def test_resize_when_pages_run_out():
    """The first row that cannot have all gets none, nor do those behind it."""
    pool, state = both(10, 5, 8, 4)
    for lens in ([4, 8, 12, 0, 0], [4, 8, 32, 4, 4], [4, 8, 12, 4, 0], [0, 32, 0, 0, 4],
                 [32, 32, 4, 4, 4], [0] * 5, [0, 0, 40, 0, 0], [33, 4, 32, 1, 0]):
        assert dspark.dspark_resize_pages(*state, i32(lens), 4).tolist() == pool.resize(lens)
        same(pool, state)


@pytest.mark.parametrize("pages", [37, 30000])
def test_fork(pages):
    rng = random.Random(pages)
    rows, width, page = 40, 12, 16
    pool, state = both(pages, rows, width, page)
    for turn in range(8):
        lens = [rng.randint(0, width * page) if b < 6 else n * page
                for b, n in enumerate(pool.held)]
        assert dspark.dspark_resize_pages(*state, i32(lens), page).tolist() == pool.resize(lens)
        n = rng.randint(1, 30)
        src = [rng.randrange(6) for _ in range(n)]
        dst = [rng.randint(6, rows - 1) for _ in range(n)]  # some of them twice
        at = [rng.randint(0, width * page + 9) if rng.random() < 0.7 else rng.randint(0, 12) * page
              for _ in range(rows)]
        at[2] = -4
        got = dspark.dspark_fork_pages(*state, i32(src), i32(dst), i32(at), page)
        want = pool.fork(src, dst, at)
        assert list(zip(*[x.tolist() for x in got])) == want
        # entries past what a row holds are -1 or what the row held before
        table, held, refs = state
        assert held.tolist() == pool.held and refs.tolist() == pool.refs
        assert table.tolist() == pool.table


def test_forks_that_cannot_be():
    """Rows outside the table, a target twice, a target that is a source, onto itself."""
    pool, state = both(50, 6, 4, 8)
    lens = [30, 9, 0, 0, 5, 0]
    dspark.dspark_resize_pages(*state, i32(lens), 8)
    pool.resize(lens)
    src, dst = [0, 0, -1, 1, 1, 6, 0, 2, 4], [2, 2, 3, 0, 1, 3, 6, 5, 3]
    got = dspark.dspark_fork_pages(*state, i32(src), i32(dst), i32(lens), 8)
    want = pool.fork(src, dst, lens)
    assert list(zip(*[x.tolist() for x in got])) == want
    assert [w[3] for w in want] == [0, 0, 0, 0, 0, 0, 0, 1, 0]
    same(pool, state)


def test_many_forks_of_one_row():
    pool, state = both(9000, 3001, 9, 4)
    lens = [33] + [0] * 3000
    dspark.dspark_resize_pages(*state, i32(lens), 4)
    pool.resize(lens)
    src, dst = [0] * 3000, list(range(1, 3001))
    for _ in range(2):  # the second time over rows that hold pages
        got = dspark.dspark_fork_pages(*state, i32(src), i32(dst), i32(lens), 4)
        assert list(zip(*[x.tolist() for x in got])) == pool.fork(src, dst, lens)
        same(pool, state)
    assert state[2][:8].tolist() == [3001] * 8


def test_a_graph_of_resize_and_fork():
    pool, state = both(400, 20, 10, 8)
    lens, more = i32([0] * 20), i32([0] * 20)
    src, dst = i32([0, 1]), i32([10, 11])
    granted = torch.zeros_like(lens)
    out = tuple(torch.zeros_like(src) for _ in range(4))

    def body():
        dspark.dspark_resize_pages(*state, lens, 8, granted=granted)
        dspark.dspark_fork_pages(*state, src, dst, more, 8, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    rng = random.Random(4)
    for _ in range(5):
        a, f = [rng.randint(0, 80) for _ in range(20)], [rng.randint(0, 80) for _ in range(20)]
        lens.copy_(i32(a))
        more.copy_(i32(f))
        graph.replay()
        torch.cuda.synchronize()
        assert granted.tolist() == pool.resize(a)
        assert list(zip(*[x.tolist() for x in out])) == pool.fork([0, 1], [10, 11], f)
        same(pool, state)


@pytest.mark.parametrize("Hkv,D,page,layout,offset", [
    (2, 128, 16, "page_head", 0), (3, 64, 7, "page_slot", 0), (1, 8, 1, "page_head", 0),
    (4, 72, 16, "page_slot", 2), (2, 20, 32, "page_head", 0), (2, 1, 16, "page_head", 0)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_copy(Hkv, D, page, layout, offset, cache):
    pages = 20
    k, v = pools(3, pages, Hkv, page, D, cache, 9, layout, offset)
    for slots in (None, [0, page, page // 2, -3, page + 9, 1, 1, 1]):
        gk, gv = on_device(k, cache, offset), on_device(v, cache, offset)
        src, dst = [3, 3, 4, 5, 6, -1, 7, 8], [10, 11, 12, 13, 14, 15, pages, 8]
        dspark.dspark_copy_pages(gk, gv, i32(src), i32(dst), None if slots is None else i32(slots))
        for x, g in ((k.clone(), gk), (v.clone(), gv)):
            for i, (a, z) in enumerate(zip(src, dst)):
                n = page if slots is None else min(max(slots[i], 0), page)
                if 0 <= a < pages and 0 <= z < pages:
                    x[:, z, :, :n] = x[:, a, :, :n].clone()
            assert same_bytes(g, x)


def test_copy_in_a_pool_past_32_bits():
    """Layers whose bytes lie past 2^32."""
    pages = 5 * 2 ** 30 // (2 * 2 * 16 * 128)
    k = torch.zeros((2, pages, 2, 16, 128), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[:, pages - 1] = 3
    v[:, pages - 1] = 5
    dspark.dspark_copy_pages(k, v, i32([pages - 1]), i32([pages - 3]), i32([9]))
    dspark.dspark_move_kv(k, v, i32([[0, 12]]), i32([1]), i32([1]), i32([[pages - 1]]))
    for x, value in ((k, 3), (v, 5)):
        assert bool((x[:, pages - 3, :, :9] == value).all())
        assert float(x[:, pages - 3, :, 9:].abs().max()) == 0.0
        assert float(x[:, :pages - 3].abs().max()) == 0.0
        assert bool((x[:, pages - 1] == value).all())
    del k, v, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [1, 16, 17, 40])
@pytest.mark.parametrize("width", [200, 256, 257, 700])
def test_forks_of_long_rows(n, width):
    """As many forks as one launch takes and more, rows of as many pages and more."""
    pool, state = both(3 * width + 2 * n + 9, n + 3, width, 4)
    lens = [4 * width - 1, 2 * width, 4 * width - 6] + [0] * n
    dspark.dspark_resize_pages(*state, i32(lens), 4)
    pool.resize(lens)
    src, dst = [i % 3 for i in range(n)], list(range(3, n + 3))
    for at in (lens, [4 * width, 9, 4 * width - 6] + [0] * n):
        got = dspark.dspark_fork_pages(*state, i32(src), i32(dst), i32(at), 4)
        assert list(zip(*[x.tolist() for x in got])) == pool.fork(src, dst, at)
        same(pool, state)
