"""Attention of drafted trees and of windows with first positions that stay visible
against its 64-bit definition (needs an MI355X): trees from one node to hundreds,
any masks, head groups, types, page sizes, windows and sinks, rows that see nothing,
values that are not finite, graph replays."""
import random

import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
import tree_ref as ref
from test_gpu_attention import SCALES, make, pools
from test_gpu_tree import forest, i32

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def words_of(bits, words):
    return [[ref.signed(x >> (32 * w) & 0xFFFFFFFF) for w in range(words)] for x in bits]


def tree(c, seed, window=0, sinks=0, branch=0.5):
    """Depths and masks of a tree on every request of a case, kept in it."""
    rows = [b - a for a, b in zip(c["cu"], c["cu"][1:])]
    parents = forest(rows, seed, branch)
    words = -(-max(rows) // 32)
    m = ref.masks(parents, c["cu"], max(rows), words, c["ctx"], window, sinks)
    fill = c["cap"] - len(m)
    c["depths"] = [m[r][0] for r in range(len(m))] + [0] * fill
    c["bits"] = [sum(w << 32 * i for i, w in enumerate(m[r][1])) for r in range(len(m))] + [0] * fill
    c["words"] = words
    return c


def call(c, kc, vc, out, **kw):
    if "bits" in c:
        kw.update(depths=i32(c["depths"]), masks=i32(words_of(c["bits"], c["words"])))
    return dspark.dspark_tree_attention(c["q"].to(DEV)[:, :, :c["D"]], kc, vc, i32(c["cu"]),
                                        i32(c["ctx"]), c["table"].to(DEV), c["max_rows"], out=out,
                                        **kw)


def check(c, **kw):
    kc, vc = pools(c, "cpu")
    out = torch.randn((c["cap"], c["Hq"], c["D"])).bfloat16()
    want, tol = ref.attend(c["q"][:, :, :c["D"]], kc, vc, c["cu"], c["ctx"], c["table"],
                           c["max_rows"], c.get("depths"), c.get("bits"), out=out, **kw)
    got = call(c, *pools(c, DEV), out.to(DEV), **kw)
    torch.cuda.synchronize()
    got = got.cpu().double()
    assert not bool(torch.isnan(got).any())
    off = (got - want).abs()
    bad = off > tol
    assert not bool(bad.any()), (int(bad.sum()), float(off.max()),
                                 [int(i) for i in bad.nonzero()[0]])
    return got


@pytest.mark.parametrize("Hq,Hkv,D,page", [
    (8, 2, 128, 16), (5, 1, 64, 32), (6, 3, 64, 64), (4, 4, 128, 128), (8, 1, 128, 64),
    (3, 1, 80, 16), (2, 1, 256, 16), (2, 2, 8, 16), (4, 2, 96, 24), (2, 1, 128, 1), (4, 1, 64, 7)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_trees(Hq, Hkv, D, page, cache):
    c = make([1, 17, 4, 0, 32, 9], [0, 300, 63, 10, 1, 129], Hq, Hkv, D, page, cache, seed=D + Hq)
    check(tree(c, D), **SCALES[cache])


@pytest.mark.parametrize("ctx", [0, 1, 31, 32, 33, 63, 64, 127, 128, 1000, 4097])
@pytest.mark.parametrize("n", [1, 2, 33, 64])
def test_trees_around_tile_borders(ctx, n):
    check(tree(make([n], [ctx], 4, 2, 128, 16, seed=ctx), n))
    check(tree(make([n], [ctx], 4, 2, 64, 16, "e4m3", seed=ctx), n), **SCALES["e4m3"])


@pytest.mark.parametrize("n", [65, 96, 97, 200, 300])
@pytest.mark.parametrize("D,G", [(128, 1), (64, 4)])
def test_trees_of_several_words(n, D, G):
    check(tree(make([n, 3, n // 2], [70, 500, 0], 2 * G, 2, D, 16, seed=n), n))


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (2, 5), (40, 1), (40, 33), (200, 64),
                                          (64, 65), (64, 300), (1000, 7), (1, 1000)])
@pytest.mark.parametrize("D", [64, 128])
def test_trees_in_windows(window, sinks, D):
    kw = dict(window=window, sinks=sinks)
    c = make([24, 1, 40, 3, 9], [500, 2000, 7, 0, 130], 4, 2, D, 32, seed=window + sinks)
    check(tree(c, D, branch=0.2, **kw), **kw)
    c = make([5, 30], [700, 63], 4, 2, D, 16, "e4m3", seed=window)
    check(tree(c, D, branch=0.2, **kw), **kw, **SCALES["e4m3"])


@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 64), (16, 4), (100, 33), (64, 64), (64, 65),
                                          (100, 200), (300, 128), (1000, 4), (0, 9), (70, 100000)])
@pytest.mark.parametrize("D", [64, 128, 96, 136])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_chains_with_sinks(window, sinks, D, cache):
    kw = dict(window=window, sinks=sinks)
    c = make([17, 1, 5, 140, 1, 0], [500, 2000, 7, 90, 64, 3], 4, 2, D, 32, cache, seed=window)
    check(c, **kw, **SCALES[cache])
    check(make([1, 1, 2], [1700, 3, 300], 4, 2, D, 16, cache, seed=window), **kw, **SCALES[cache])


def test_prompts_with_sinks():
    for rows, ctx in (([150, 1, 64, 257], [0, 0, 0, 0]), ([130, 300], [333, 1001])):
        for window, sinks in ((64, 4), (100, 16), (17, 130)):
            check(make(rows, ctx, 8, 2, 128, 16, seed=window), window=window, sinks=sinks)
            check(make(rows, ctx, 3, 1, 64, 32, seed=window), window=window, sinks=sinks)


def test_a_chain_without_sinks_is_dspark_verify_attention():
    """By definition: either lies within the bound of the 64-bit result."""
    for rows in ([17, 1, 5], [100, 300, 2]):
        c = make(rows, [3000, 900, 40], 8, 2, 128, 16, seed=10)
        kc, vc = pools(c, DEV)
        for window in (0, 50, 2000):
            check(c, window=window)
            out = torch.randn((c["cap"], 8, 128)).bfloat16()
            want, tol = ref.attend(c["q"], c["kc"], c["vc"], c["cu"], c["ctx"], c["table"],
                                   c["max_rows"], window=window, out=out)
            got = dspark.dspark_verify_attention(c["q"].to(DEV), kc, vc, i32(c["cu"]), i32(c["ctx"]),
                                                 c["table"].to(DEV), c["max_rows"], window=window,
                                                 out=out.to(DEV))
            assert bool(((got.cpu().double() - want).abs() <= tol).all())


def any_masks(c, seed, density=0.5, words=None):
    """Bits at random: later rows, rows past the request's, rows that see none."""
    rng = random.Random(seed)
    c["words"] = words or -(-c["max_rows"] // 32)
    some = lambda: sum((rng.random() < density) << i for i in range(32 * c["words"]))  # noqa: E731
    c["bits"] = [0 if rng.random() < 0.2 else some() for _ in range(c["cap"])]
    c["depths"] = [rng.randint(-2, 40) for _ in range(c["cap"])]
    return c


@pytest.mark.parametrize("D", [64, 128, 136])
@pytest.mark.parametrize("rows,ctx", [([20, 33, 1, 64], [0, 100, 0, 31]), ([150, 40], [0, 70]),
                                      ([5, 9], [0, 0])])
def test_any_masks(rows, ctx, D):
    """Rows without a bit and without a context give zeros."""
    for words in (None, 7):
        c = any_masks(make(rows, ctx, 4, 2, D, 16, seed=D), D, words=words)
        got = check(c)
        for b, n in enumerate(rows):
            for j in range(n):
                if ctx[b] == 0 and c["bits"][c["cu"][b] + j] & ((1 << n) - 1) == 0:
                    assert float(got[c["cu"][b] + j].abs().max()) == 0.0
        check(c, window=9, sinks=3)
        check(any_masks(c, D + 1, density=0.03), window=40)


def test_masks_of_rows_past_max_rows():
    c = any_masks(make([9, 40, 3], [50, 0, 5], 4, 2, 128, 16, seed=1), 2, words=2)
    c["max_rows"] = 6
    check(c)
    c["table"] = c["table"][:, :2].contiguous()  # and a table shorter than the rows
    check(c)


@pytest.mark.parametrize("rows", [[1, 1, 1, 1], [17, 3, 17, 3], [100, 2, 90, 3]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 40)])
def test_pages_the_table_does_not_name(rows, window, sinks):
    c = make(rows, [100, 100, 5, 200], 4, 2, 128, 16, seed=2)
    pages = c["kc"].shape[0]
    c["table"][0, 2] = -1
    c["table"][1, :] = pages          # nothing to see: zeros
    c["table"][2, 0] = pages + 5
    c["table"][3, 3:6] = -9
    kw = dict(window=window, sinks=sinks)
    check(c, **kw)
    got = check(tree(c, 3, **kw), **kw)
    r = c["cu"][1]
    assert float(got[r:r + rows[1]].abs().max()) == 0.0


@pytest.mark.parametrize("D", [64, 128, 96, 136])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,ctx,window,sinks", [
    ([17, 1, 9], [300, 63, 5], 0, 0), ([24, 40], [100, 0], 30, 5), ([90, 70], [0, 200], 20, 40)])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(D, cache, rows, ctx, window,
                                                                      sinks):
    """In a node that some rows see, in a position that the window has passed, and
    in one that the sinks keep."""
    kw = dict(window=window, sinks=sinks)
    c = tree(make(rows, ctx, 4, 2, D, 16, cache, seed=12), 5, **kw)
    clean = check(c, **kw, **SCALES[cache])
    bad = float("nan") if cache == "e4m3" else float("inf")
    hits = [[ctx[b] + n // 2 for b, n in enumerate(rows)], [ctx[b] // 2 for b in range(len(rows))],
            [0] * len(rows)]
    for at in hits:
        for pool in ("vc", "kc"):
            x = dict(c, kc=c["kc"].clone(), vc=c["vc"].clone())
            for b, t in enumerate(at):
                page = x[pool][int(c["table"][b, t // 16])].float()
                page[:, t % 16, 3::7] = bad if pool == "vc" else float("nan")
                raw = page.to(x[pool].dtype).view(torch.uint8)
                x[pool].view(torch.uint8)[int(c["table"][b, t // 16])] = raw
            out = torch.zeros((c["cap"], c["Hq"], D), dtype=torch.bfloat16, device=DEV)
            got = call(x, *pools(x, DEV), out, **kw, **SCALES[cache]).cpu().double()
            for b, n in enumerate(rows):
                for j in range(n):
                    r = c["cu"][b] + j
                    if at[b] in ref.seen(ctx[b], n, j, c["depths"][r], c["bits"][r], window, sinks):
                        assert not bool(got[r, :, 3::7].isfinite().any()), (b, j)
                    else:
                        assert torch.equal(got[r], clean[r]), (b, j)


def test_what_is_not_seen_may_hold_anything():
    """NaN in every slot that no row of its request sees."""
    kw = dict(window=30, sinks=5)
    c = tree(make([12, 1, 40], [90, 70, 300], 4, 2, 128, 16, seed=3), 4, **kw)
    clean = check(c, **kw)
    live = torch.zeros(c["kc"].shape[0], 16, dtype=torch.bool)
    for b in range(3):
        n = c["cu"][b + 1] - c["cu"][b]
        for j in range(n):
            r = c["cu"][b] + j
            for t in ref.seen(c["ctx"][b], n, j, c["depths"][r], c["bits"][r], **kw):
                live[int(c["table"][b, t // 16]), t % 16] = True
    for x, bad in ((c["kc"], float("nan")), (c["vc"], float("inf"))):
        x.copy_(torch.where(live[:, None, :, None], x, torch.full_like(x, bad)))
    out = torch.zeros((c["cap"], c["Hq"], c["D"]), dtype=torch.bfloat16, device=DEV)
    got = call(c, *pools(c, DEV), out, **kw).cpu().double()
    assert torch.equal(got[:c["cu"][-1]], clean[:c["cu"][-1]])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_other_axis_order_and_strided_queries(D, cache):
    c = make([30, 1, 40], [40, 100, 0], 8, 2, D, 16, cache, seed=1, layout="page_slot", q_pad=64)
    check(tree(c, D), **SCALES[cache])
    check(tree(c, D, 20, 6), window=20, sinks=6, **SCALES[cache])


def test_long_contexts_split_over_the_device():
    check(tree(make([40], [30011], 4, 1, 128, 16, "e4m3", seed=7), 1), **SCALES["e4m3"])
    check(tree(make([70, 3], [20000, 9], 2, 1, 64, 64, seed=8), 1))
    check(make([1, 2], [30000, 20000], 4, 2, 128, 16, seed=8), window=9000, sinks=5000)


def test_many_requests():
    rng = random.Random(9)
    rows = [rng.choice((0, 1, 2, 5, 17, 30)) for _ in range(700)]
    ctx = [rng.randint(0, 90) for _ in rows]
    c = make(rows, ctx, 2, 1, 64, 16, seed=9)
    check(tree(c, 9, 20, 3), window=20, sinks=3)


def test_lengths_the_kernels_bound():
    c = make([4, 6, 5], [-3, 60, 33], 4, 2, 128, 16, seed=6)
    check(tree(c, 2))
    check(tree(c, 2, 8, 2), window=8, sinks=2)
    check(make([4, 6, 5], [-3, 60, 33], 4, 2, 128, 16, seed=6), window=8, sinks=2)


def test_large_scores_and_scales_of_either_sign():
    c = tree(make([20, 1], [300, 900], 4, 2, 128, 16, seed=4, spread=100.0), 4)
    check(c)
    check(c, scale=-0.05)
    check(tree(make([9, 40], [300, 10], 4, 2, 64, 16, seed=5), 5), scale=0.0)


@pytest.mark.parametrize("D", [8, 24, 40, 72, 112, 192])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_other_head_sizes(D, cache):
    c = make([30, 1, 40, 17], [40, 300, 0, 129], 4, 2, D, 16, cache, seed=D)
    check(tree(c, D, 25, 6), window=25, sinks=6, **SCALES[cache])
    check(tree(make([70, 1], [90, 5], 4, 1, D, 7, cache, seed=D, layout="page_slot"), D),
          **SCALES[cache])


def test_graph_replays_with_new_trees():
    """One captured step: masks, then two layers, one of them with a window and sinks."""
    rows = [30, 1, 20, 3]
    c = make(rows, [900, 2000, 40, 0], 8, 2, 128, 16, seed=11)
    kc, vc = pools(c, DEV)
    q, cu, ctx, table = c["q"].to(DEV), i32(c["cu"]), i32(c["ctx"]), c["table"].to(DEV)
    parents = i32(forest(rows, 1) + [0] * (c["cap"] - c["cu"][-1]))
    a, b = (torch.zeros((c["cap"], 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def body():
        for out, window, sinks in ((a, 0, 0), (b, 40, 4)):
            depths, masks = dspark.dspark_tree_masks(parents, cu, 30, ctx_lens=ctx, window=window,
                                                     sinks=sinks)
            dspark.dspark_tree_attention(q, kc, vc, cu, ctx, table, 30, depths=depths, masks=masks,
                                         window=window, sinks=sinks, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for turn, (rows, lens) in enumerate((([30, 1, 20, 3], [900, 2000, 40, 0]),
                                         ([1, 1, 1, 1], [5, 1000, 44, 2]),
                                         ([3, 20, 17, 5], [20, 7, 28, 1])) * 2):
        case = dict(c, cu=[0], ctx=lens)
        for n in rows:
            case["cu"] = case["cu"] + [case["cu"][-1] + n]
        case["max_rows"] = 30
        tree_ = forest(rows, turn)
        parents[:len(tree_)] = i32(tree_)
        cu.copy_(i32(case["cu"]))
        ctx.copy_(i32(lens))
        a.fill_(7)
        b.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone(), b.clone()]
        a.fill_(7)
        b.fill_(7)
        body()
        torch.cuda.synchronize()
        assert torch.equal(got[0], a) and torch.equal(got[1], b)
        for out, window, sinks in ((a, 0, 0), (b, 40, 4)):
            m = ref.masks(tree_, case["cu"], 30, 1, lens, window, sinks)
            depths = [m[r][0] for r in range(len(m))]
            bits = [m[r][1][0] for r in range(len(m))]
            want, tol = ref.attend(c["q"], c["kc"], c["vc"], case["cu"], lens, c["table"], 30,
                                   depths, bits, window, sinks,
                                   out=torch.full(out.shape, 7.0).bfloat16())
            assert bool(((out.cpu().double() - want).abs() <= tol).all())


def test_both_attentions_share_a_workspace():
    """Chains and trees in turn, split and joined: each as before."""
    c = make([17, 1, 5], [3000, 900, 40], 8, 2, 128, 16, seed=10)
    t = tree(make([30, 60], [2000, 9000], 8, 2, 128, 16, seed=11), 1)
    args = (c["q"].to(DEV), *pools(c, DEV), i32(c["cu"]), i32(c["ctx"]), c["table"].to(DEV), 17)
    first = dspark.dspark_verify_attention(*args)[:23].clone()
    for _ in range(3):
        check(t)
        check(c, window=500, sinks=9)
        check(c)
        assert torch.equal(dspark.dspark_verify_attention(*args)[:23], first)


def test_requests_without_rows_among_few_units():
    """Their units are none: nothing is joined for them, whatever the workspace held."""
    big = tree(make([60, 64], [9000, 4000], 8, 2, 128, 16, seed=1), 1)
    for rows in ([0, 9], [5, 0, 0], [0, 0], [64, 0, 1]):
        check(big)
        c = make(rows, [700] * len(rows), 8, 2, 128, 16, seed=2)
        c["max_rows"] = 64
        check(tree(c, 2) if any(rows) else c, window=300, sinks=2)
    wide = make([500, 0, 3], [300, 9, 5000], 4, 1, 64, 16, seed=3)
    check(wide)
    check(make([3, 0, 500], [9000, 9, 20], 4, 1, 64, 16, seed=4))
    check(wide, window=100, sinks=70)


def test_repeats_are_equal_and_on_another_stream():
    c = tree(make([40, 1, 5], [3000, 900, 40], 8, 2, 128, 16, seed=10), 3)
    kc, vc = pools(c, DEV)
    a = call(c, kc, vc, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = call(c, kc, vc, None)
    torch.cuda.synchronize()
    assert torch.equal(a[:c["cu"][-1]], b[:c["cu"][-1]])


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1),
                                          (3, 2 ** 31 - 1), (2 ** 31 - 1, 5)])
def test_the_largest_windows_and_sinks(window, sinks):
    kw = dict(window=window, sinks=sinks)
    c = make([20, 1, 90], [0, 130, 60], 4, 2, 128, 16, seed=2)
    check(c, **kw)
    check(tree(c, 3, **kw), **kw)
    check(make([9], [40], 2, 1, 136, 16, seed=2), **kw)


def test_heads_in_groups_past_a_block():
    """One row of a key-value head fills more than a block of query rows."""
    check(tree(make([5, 1, 3], [40, 100, 0], 300, 1, 64, 16, seed=4), 2))
    check(make([2, 1], [90, 700], 130, 1, 64, 16, seed=4), window=60, sinks=70)


def test_equal_units_are_not_cut():
    """As many units as workgroups and more, all alike, in a window: whole ones each."""
    for n, B, Hkv in ((1, 128, 8), (3, 70, 8), (2, 300, 2)):
        c = make([n] * B, [90 + b % 7 for b in range(B)], Hkv, Hkv, 64, 16, seed=B)
        check(c, window=64, sinks=4)
        check(tree(c, 1, 64, 4), window=64, sinks=4)


def test_two_calls_at_once_with_a_workspace_each():
    """Calls on two streams, their contexts split over the device and joined."""
    cases = [tree(make([40, 1], [3000, 9000], 8, 2, 128, 16, seed=s), s) for s in (1, 2)]
    args = [(c["q"].to(DEV), *pools(c, DEV), i32(c["cu"]), i32(c["ctx"]), c["table"].to(DEV), 40)
            for c in cases]
    kws = [dict(depths=i32(c["depths"]), masks=i32(words_of(c["bits"], c["words"]))) for c in cases]
    want = [dspark.dspark_tree_attention(*a, **k)[:41].clone() for a, k in zip(args, kws)]
    need = dspark.dspark_attention_workspace_bytes(2, 40, 8, 2, 128)
    ws = [torch.zeros(need, dtype=torch.uint8, device=DEV) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(dspark.dspark_tree_attention(*args[i], ws=ws[i], **kws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x[:41], want[i]) for x in got[i])


def test_two_graphs_share_a_workspace():
    """Graphs of calls of different sizes, replayed in turn with eager calls between."""
    cases = [tree(make([n, 3], [2500, 700], 8, 2, 128, 16, seed=n), n) for n in (30, 64)]
    graphs = []
    for c in cases:
        args = (c["q"].to(DEV), *pools(c, DEV), i32(c["cu"]), i32(c["ctx"]), c["table"].to(DEV),
                c["max_rows"])
        kw = dict(depths=i32(c["depths"]), masks=i32(words_of(c["bits"], c["words"])))
        want = dspark.dspark_tree_attention(*args, **kw).clone()
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dspark.dspark_tree_attention(*args, out=out, **kw)
        graphs.append((graph, args, kw, out, want, c["cu"][-1]))
    for _ in range(3):
        for graph, args, kw, out, want, n in graphs:
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[:n], want[:n])
            assert torch.equal(dspark.dspark_tree_attention(*args, **kw)[:n], want[:n])
