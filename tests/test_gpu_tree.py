"""Drafted trees against their plain definitions (needs an MI355X): the ancestors
of every node, the append of nodes at their own positions, the walk down the tree
by the target's choices, and the move of the accepted keys and values."""
import random

import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
import tree_ref as ref
from test_gpu_append import make, views

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts(rows):
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    return cu


def forest(rows, seed, branch=0.5):
    rng = random.Random(seed)
    return sum((ref.some_tree(rng, n, branch) for n in rows if n), [])


# ---------------------------------------------------------------------- masks

@pytest.mark.parametrize("rows", [[1], [0, 1, 0], [31, 32, 33, 64, 65, 1], [200, 3], [1024, 5]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 0), (2, 4), (5, 1000), (1, 3)])
def test_masks(rows, window, sinks):
    cu, parents = starts(rows), forest(rows, sum(rows), 0.3)
    ctx = [random.Random(b).choice((0, 1, 5, 100)) for b in range(len(rows))]
    cap = cu[-1] + 2
    words = -(-max(rows) // 32)
    depths = torch.full((cap,), -7, dtype=torch.int32, device=DEV)
    masks = torch.full((cap, words), -7, dtype=torch.int32, device=DEV)
    dspark.dspark_tree_masks(i32(parents + [0, 0]), i32(cu), max(rows), ctx_lens=i32(ctx),
                             window=window, sinks=sinks, out=(depths, masks))
    want = ref.masks(parents, cu, max(rows), words, ctx, window, sinks)
    depths, masks = depths.tolist(), masks.tolist()
    for r in range(cap):
        depth, bits = want.get(r, (-7, None))
        assert depths[r] == depth, r
        assert masks[r] == ([ref.signed(w) for w in bits] if bits else [-7] * words), r


def test_masks_of_forests_and_of_parents_that_are_none():
    """Roots beside row 0; parents that are not below their rows are roots too."""
    parents = [5, 0, -1, 2, 4, 900, 5, -9, 6]
    depths, masks = dspark.dspark_tree_masks(i32(parents), i32([0, 9]), 9)
    assert depths.tolist() == [0, 1, 0, 1, 0, 0, 1, 0, 2]
    assert masks.flatten().tolist() == [1, 3, 4, 12, 16, 32, 96, 128, 32 + 64 + 256]


def test_masks_of_more_words_than_rows_need_and_rows_past_max_rows():
    parents = [-1, 0, 1, 1, 0]
    out = (torch.full((5,), 9, dtype=torch.int32, device=DEV),
           torch.full((5, 3), 9, dtype=torch.int32, device=DEV))
    dspark.dspark_tree_masks(i32(parents), i32([0, 5]), 3, out=out)
    assert out[0].tolist() == [0, 1, 2, 9, 9]
    assert out[1].tolist() == [[1, 0, 0], [3, 0, 0], [7, 0, 0], [9] * 3, [9] * 3]


def test_masks_of_lengths_that_the_kernels_bound():
    """cu_seqlens past the rows, or falling, are clamped."""
    depths, masks = dspark.dspark_tree_masks(i32([-1, 0, 0]), i32([0, 900, 2]), 8)
    assert depths.tolist() == [0, 1, 1] and masks.flatten().tolist() == [1, 3, 5]


def test_masks_of_many_requests():
    rows = [1 + b % 3 for b in range(70000)]
    cu = starts(rows)
    parents = sum(([-1, 0, 0][:n] for n in rows), [])
    depths, masks = dspark.dspark_tree_masks(i32(parents), i32(cu), 3)
    assert depths.tolist() == sum(([0, 1, 1][:n] for n in rows), [])
    assert masks.flatten().tolist() == sum(([1, 3, 5][:n] for n in rows), [])


# --------------------------------------------------------------------- append

@pytest.mark.parametrize("Hq,Hkv,D,page,rot", [(8, 2, 128, 16, 128), (5, 1, 64, 32, 32),
                                               (4, 4, 80, 7, 40), (2, 1, 24, 16, 10)])
@pytest.mark.parametrize("cache,interleaved", [("bf16", False), ("bf16", True), ("e4m3", True)])
def test_append(Hq, Hkv, D, page, rot, cache, interleaved):
    rows = [9, 1, 0, 33, 4]
    c = make(len(rows), rows, Hq, Hkv, D, page, cache, rot=rot, seed=Hq + D, holes=True)
    depths = [ref.lineage(t, j) for n in rows if n
              for t in [ref.some_tree(random.Random(n), n)] for j in range(n)]
    depths = [len(up) - 1 for up in depths] + [0, 0]
    depths[2], depths[4] = -3, 1000  # taken as 0 and as the row's place
    kw = dict(interleaved=interleaved)
    if cache == "e4m3":
        kw.update(k_scale=0.05, v_scale=0.02)
    q, k, v, kc, vc = views(c, "cpu")
    out = torch.randn(q.shape).bfloat16()
    want, tol = ref.append(q, k, v, c["cos"], c["sin"], depths, c["cu"], c["ctx"], c["table"], kc,
                           vc, out=out, **kw)
    gq, gk, gv, gkc, gvc = views(c, DEV)
    got = dspark.dspark_append_tree_kv(gq, gk, gv, c["cos"].to(DEV), c["sin"].to(DEV), i32(depths),
                                       i32(c["cu"]), i32(c["ctx"]), c["table"].to(DEV), gkc, gvc,
                                       out=out.to(DEV), **kw)
    torch.cuda.synchronize()
    for g, w, t in zip((got, gkc, gvc), want, tol):
        off = (g.cpu().double() - w).abs()
        assert bool((off <= t).all()), float(off.max())


def test_append_of_a_chain_is_the_chains():
    rows = [5, 1, 17]
    c = make(3, rows, 8, 2, 128, 16, seed=3)
    depths = [j for n in rows for j in range(n)] + [0, 0]
    a, b = views(c, DEV), views(c, DEV)
    common = (i32(c["cu"]), i32(c["ctx"]), c["table"].to(DEV))
    x = dspark.dspark_append_kv(*a[:3], c["cos"].to(DEV), c["sin"].to(DEV), *common, *a[3:])
    y = dspark.dspark_append_tree_kv(*b[:3], c["cos"].to(DEV), c["sin"].to(DEV), i32(depths),
                                     *common, *b[3:])
    n = c["cu"][-1]
    assert torch.equal(x[:n], y[:n]) and torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])


# --------------------------------------------------------------------- accept

def tree_case(rows, seed, follow=0.8, vocabulary=50):
    rng = random.Random(seed)
    cu, parents = starts(rows), forest(rows, seed)
    tokens = [rng.randrange(vocabulary) for _ in range(cu[-1])]
    choice = [rng.randrange(vocabulary) for _ in range(cu[-1])]
    for b, n in enumerate(rows):  # the choices follow some branch for a while
        at = rng.randrange(n) if n else 0
        while at > 0:
            p = parents[cu[b] + at]
            if rng.random() < follow:
                choice[cu[b] + p] = tokens[cu[b] + at]
            at = p
    return cu, parents, tokens, choice


def check_accept(cu, parents, tokens, choice, max_rows, width):
    got = dspark.dspark_tree_accept(i32(choice), i32(tokens), i32(parents), i32(cu), max_rows, width)
    for g, w in zip(got, ref.accept(choice, tokens, parents, cu, max_rows, width)):
        assert g.tolist() == w
    return got


@pytest.mark.parametrize("rows", [[1], [2, 0, 5], [64, 65, 63, 1, 128, 129], [1024, 7], [17] * 300])
@pytest.mark.parametrize("width", [1, 2, 9, 70])
def test_accept(rows, width):
    check_accept(*tree_case(rows, sum(rows)), max(rows), width)
    check_accept(*tree_case(rows, sum(rows) + 1, vocabulary=2), max(rows), width)


def test_accept_takes_the_lowest_of_equal_children():
    parents, tokens = [-1, 0, 0, 2, 1, 2], [9, 4, 4, 7, 7, 7]
    acc, bonus, path = check_accept([0, 6], parents, tokens, [4, 7, 7, 1, 2, 3], 6, 4)
    assert path.tolist() == [[0, 1, 4, -1]] and bonus.tolist() == [2] and acc.tolist() == [2]


def test_accept_on_a_chain_is_dspark_accept():
    B, g, V = 9, 6, 300
    gen = torch.Generator(device=DEV).manual_seed(1)
    logits = torch.randn((B * (g + 1), V), generator=gen, device=DEV).bfloat16()
    tokens = logits.view(B, g + 1, V).argmax(-1).roll(1, 1).to(torch.int32).contiguous()
    tokens[::2, 3] = 5
    cu = i32([b * (g + 1) for b in range(B + 1)])
    choice, acc, bonus = dspark.dspark_accept(logits, None, cu, tokens)
    parents = i32([j - 1 for j in range(g + 1)] * B)
    a, z, path = dspark.dspark_tree_accept(choice, tokens.view(-1), parents, cu, g + 1, g + 1)
    assert torch.equal(a, acc) and torch.equal(z, bonus)
    for b, n in enumerate(acc.tolist()):
        assert path[b].tolist() == list(range(n + 1)) + [-1] * (g - n)


def test_accept_leaves_out_rows_past_max_rows_and_bounds_lengths():
    cu, parents, tokens, choice = tree_case([40, 12], 3, follow=1.0)
    check_accept(cu, parents, tokens, choice, 10, 12)
    got = dspark.dspark_tree_accept(i32(choice), i32(tokens), i32(parents), i32([0, 90, 52]), 64, 5)
    assert got[0].shape == (2,) and got[1][1] == -1 and got[2][1].tolist() == [-1] * 5


# ----------------------------------------------------------------------- move

def pools(layers, pages, Hkv, page, D, cache, seed, layout="page_head", offset=0):
    gen = torch.Generator().manual_seed(seed)
    shape = {"page_head": (layers, pages, Hkv, page, D), "page_slot": (layers, pages, page, Hkv, D)}
    n = layers * pages * Hkv * page * D
    out = []
    for _ in range(2):
        raw = torch.randint(0, 256, (offset + n * (1 if cache == "e4m3" else 2),), generator=gen,
                            dtype=torch.uint8)
        x = raw[offset:].view(torch.uint8 if cache == "e4m3" else torch.int16).view(shape[layout])
        out.append(x.transpose(2, 3) if layout == "page_slot" else x)
    return out


def on_device(x, cache, offset=0):
    """The pool's bytes on the GPU, `offset` bytes off the allocation's start."""
    axes = x.transpose(2, 3) if not x.is_contiguous() else x
    flat = axes.contiguous().view(torch.uint8).reshape(-1)
    raw = torch.zeros(flat.numel() + offset, dtype=torch.uint8, device=DEV)
    raw[offset:] = flat.to(DEV)
    y = raw[offset:].view(torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16).view(axes.shape)
    return y.transpose(2, 3) if not x.is_contiguous() else y


def same_bytes(got, want):
    got = got.view(torch.uint8 if got.dtype == torch.float8_e4m3fn else torch.int16)
    return torch.equal(got.cpu(), want)


@pytest.mark.parametrize("Hkv,D,page,layout,offset", [
    (2, 128, 16, "page_head", 0), (3, 64, 7, "page_slot", 0), (1, 8, 1, "page_head", 0),
    (4, 72, 16, "page_slot", 2), (2, 20, 32, "page_head", 0), (2, 1, 16, "page_head", 0)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_move(Hkv, D, page, layout, offset, cache):
    rows = [40, 1, 12, 30, 0, 200]
    cu, parents, tokens, choice = tree_case(rows, 5, follow=1.0)
    acc, _, paths = ref.accept(choice, tokens, parents, cu, 200, 150)
    ctx = [0, 3, 100, 17, 5, 60]
    need = [-(-(c + n) // page) for c, n in zip(ctx, rows)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).tolist()
    table = [[order.pop() for _ in range(n)] + [-1] * (max(need) + 1 - n) for n in need]
    table[2][ctx[2] // page] = pages + 1 if page < 32 else table[2][ctx[2] // page]
    k, v = pools(3, pages, Hkv, page, D, cache, 7, layout, offset)
    gk, gv = on_device(k, cache, offset), on_device(v, cache, offset)
    dspark.dspark_move_kv(gk, gv, i32(paths), i32(acc), i32(ctx), i32(table))
    for b in range(len(rows)):
        for i, j in enumerate(paths[b][1:acc[b] + 1], 1):
            old = ref.slot(table[b], ctx[b] + j, page, pages)
            new = ref.slot(table[b], ctx[b] + i, page, pages)
            if old and new:
                for x in (k, v):
                    x[:, new[0], :, new[1]] = x[:, old[0], :, old[1]].clone()
    assert same_bytes(gk, k) and same_bytes(gv, v)


def test_move_of_one_layer_and_of_lengths_that_are_bounded():
    """Four axes; an accepted count past the path; negative entries move nothing."""
    k, v = pools(1, 4, 2, 16, 64, "bf16", 8)
    gk, gv = on_device(k, "bf16")[0], on_device(v, "bf16")[0]
    dspark.dspark_move_kv(gk, gv, i32([[0, 3, -1, 9], [0, 2, 5, 7]]), i32([99, -4]), i32([-5, 20]),
                          i32([[2, 0], [3, 1]]))
    for x, g in ((k, gk), (v, gv)):
        x = x[0]
        x[2, :, 1], x[2, :, 3] = x[2, :, 3].clone(), x[2, :, 9].clone()
        assert same_bytes(g, x)
