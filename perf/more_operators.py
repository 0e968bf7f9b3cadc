"""What is measured of the operators for drafted trees and shared pages.

Four passes, as a serving loop makes them around the target's forward:

* enter: the ancestors of every drafted node (``dspark_tree_masks``), once per
  step, and the append of the nodes' keys and values, rotated by their own
  positions (``dspark_append_tree_kv``), once per layer;
* attend: attention of the packed rows over each request's pages
  (``dspark_tree_attention``): the nodes of a tree, which see the context and
  their ancestors, or rows in a chain, with a sliding window and a few first
  positions that stay visible;
* commit: the walk down the tree by the target's choices
  (``dspark_tree_accept``), then the accepted nodes' keys and values brought
  together in all layers (``dspark_move_kv``);
* fork: pages for a step's batch (``dspark_resize_pages``), continuations that
  share a prompt's pages (``dspark_fork_pages``), and copies of the pages that
  they do not share (``dspark_copy_pages``).

``run`` computes them in elementary torch operations, or, where ``own`` is true,
through the framework's entry points. ``exact`` writes their definitions out in
64 bits. Lengths and the shapes of trees belong to the case (drawn from its
``mix``); the values in the tensors come from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
E4M3_MAX = 448.0


# --------------------------------------------------------------------- cases

def _case(op, name, **kw):
    case = dict(name=name, op=op, B=1, rows="tree", least=16, most=32, depth=6, Hq=32, Hkv=8, D=128,
                page=64, ctx_lo=128, ctx_hi=4096, cache="bf16", window=0, sinks=0, mix=1)
    if op == "enter":
        case.update(rot=128, interleaved=False)
    elif op in ("commit", "fork"):
        case.update(layers=4)
        if op == "fork":
            case.update(copies=4)
    case.update(kw)
    return case


def listed():
    return [
        # one user's tree of 32 nodes enters a layer: launch latency
        _case("enter", "enter_single", least=32, ctx_lo=1000, ctx_hi=1000, page=16, mix=1),
        # a full batch of ragged trees into an 8-bit cache, half of each head rotated in pairs
        _case("enter", "enter_batch_e4m3", B=192, least=8, most=64, Hq=40, Hkv=8, page=32,
              cache="e4m3", rot=64, interleaved=True, mix=2),
        # one user's tree on an ordinary context: latency and the split over its length
        _case("attend", "tree_single", least=60, most=60, ctx_lo=4000, ctx_hi=4000, page=16, mix=3),
        # a batch of trees, groups of four
        _case("attend", "tree_batch", B=128, least=12, mix=4),
        # four long documents with whole trees of 64 nodes, an 8-bit cache
        _case("attend", "tree_long_e4m3", B=4, least=64, most=64, depth=8, ctx_lo=40000,
              ctx_hi=120000, cache="e4m3", mix=5),
        # trees in a sliding-window layer with small heads in groups of five
        _case("attend", "tree_sliding", B=64, least=8, most=24, Hq=40, D=64, page=32, ctx_lo=500,
              ctx_hi=12000, window=1024, sinks=4, mix=6),
        # plain decoding of a full batch with a window and its first tokens
        _case("attend", "sink_decode", B=256, rows="single", ctx_lo=500, ctx_hi=8000, window=1024,
              sinks=4, mix=7),
        # prompts packed together through such a layer, nothing cached before them
        _case("attend", "sink_prompts", B=4, rows="prompt", most=4096, ctx_lo=0, ctx_hi=0,
              window=1024, sinks=16, mix=8),
        # one user's tree is accepted, four layers
        _case("commit", "commit_single", least=32, ctx_lo=1000, ctx_hi=1000, page=16, mix=9),
        # a full batch of trees is accepted, all layers of a rank's part of a model
        _case("commit", "commit_batch", B=256, least=8, most=64, depth=8, layers=16, mix=10),
        # one prompt is answered four times
        _case("fork", "fork_single", ctx_lo=700, ctx_hi=700, page=16, rows="single", mix=11),
        # 32 prompts, eight answers each
        _case("fork", "fork_batch", B=32, copies=8, layers=8, ctx_lo=500, ctx_hi=8000, rows="single",
              mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _draw(rng)
        cost = work(case)  # at most that of the largest listed ones
        if cost["bytes"] <= 1.1e9 and cost["flops"] <= 3e11:
            return case


def _draw(rng):
    mix = rng.randrange(1 << 30)
    kind = rng.choice(("enter", "tree", "tree", "chain", "prompt", "commit", "fork"))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    heads = dict(Hkv=Hkv, Hq=Hkv * rng.choice((1, 2, 3, 4, 5, 8)), D=rng.choice((64, 128, 128)),
                 page=rng.choice((16, 32, 64, 128)), cache=rng.choice(("bf16", "bf16", "e4m3")))
    most = rng.randint(2, 64)
    tree = dict(least=rng.randint(1, most), most=most, depth=rng.randint(1, 10))
    window = rng.choice((0, 0, rng.randint(1, 2000), rng.randint(1, 12)))
    view = dict(window=window, sinks=rng.choice((0, rng.randint(1, 130))) if window else 0)
    if kind == "enter":
        return _case("enter", "", B=_log_int(rng, 1, 192), ctx_lo=1, ctx_hi=_log_int(rng, 64, 8000),
                     rot=rng.choice((heads["D"], heads["D"] // 2)),
                     interleaved=rng.random() < 0.5, mix=mix, **view, **tree, **heads)
    if kind in ("tree", "chain"):
        B = _log_int(rng, 1, 256)
        longest = _log_int(rng, 256, min(60000, 150000 // B))
        rows = "tree" if kind == "tree" else rng.choice(("single", "verify"))
        return _case("attend", "", B=B, rows=rows, ctx_lo=rng.choice((1, longest // 2)),
                     ctx_hi=longest, mix=mix, **view, **tree, **heads)
    if kind == "prompt":
        tree["most"] = _log_int(rng, 70, 2500)
        return _case("attend", "", B=rng.randint(1, 4), rows="prompt", ctx_lo=0,
                     ctx_hi=rng.choice((0, 300, 6000)), mix=mix, **view, **tree, **heads)
    if kind == "commit":
        return _case("commit", "", B=_log_int(rng, 1, 256), layers=rng.randint(1, 12), ctx_lo=1,
                     ctx_hi=_log_int(rng, 64, 8000), mix=mix, **tree, **heads)
    return _case("fork", "", B=_log_int(rng, 1, 32), copies=rng.randint(2, 8),
                 layers=rng.randint(1, 6), rows="single", ctx_lo=1, ctx_hi=_log_int(rng, 64, 8000),
                 mix=mix, **heads)


# ------------------------------------------- lengths, trees, tables, inputs

def _lengths(case):
    """(context, rows) of every request: tokens cached before the call, rows of the call."""
    rng = random.Random(case["mix"])
    least, most = case["least"], case["most"]
    ctx, rows = [], []
    for _ in range(case["B"]):
        lo, hi = case["ctx_lo"], case["ctx_hi"]
        ctx.append(lo if hi <= max(lo, 1) else _log_int(rng, max(lo, 1), hi))
        kind = case["rows"]
        if kind == "single":
            rows.append(1)
        elif kind == "prompt":
            rows.append(rng.randint(max(1, most // 3), most))
        elif kind == "tree":
            rows.append(rng.randint(least, most))
        else:  # a chain of drafts, cut by its confidence
            rows.append(most if rng.random() < 0.35 else 1 + min(most - 1, int(rng.expovariate(0.4))))
    return ctx, rows


def _trees(case, rows):
    """Parents of every request's nodes: the likeliest chain first, then branches off any node."""
    rng = random.Random(case["mix"] + 1)
    trees = []
    for n in rows:
        deep = min(case["depth"], n - 1)
        parents, depth = [-1], [0]
        for i in range(1, n):
            p = i - 1 if i <= deep else rng.choice([k for k in range(i) if depth[k] < deep])
            parents.append(p)
            depth.append(depth[p] + 1)
        trees.append((parents, depth))
    return trees


def _max_rows(case):
    return 1 if case["rows"] == "single" else case["most"]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cu(rows):
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    return _ints(cu)


def _normal(shape, dtype, gen, std=1.0):
    x = torch.empty(shape, dtype=torch.float32 if dtype == torch.float8_e4m3fn else dtype, device=DEV)
    x.normal_(0.0, std, generator=gen)
    return x.clamp_(-E4M3_MAX, E4M3_MAX).to(dtype) if dtype == torch.float8_e4m3fn else x


def _pools(case, pages, gen, layers=None):
    e4m3 = case["cache"] == "e4m3"
    # scales as a calibration leaves them: the values fill the 8-bit range
    dtype, k_scale, v_scale = ((torch.float8_e4m3fn, 0.03125, 0.0234375) if e4m3
                               else (torch.bfloat16, 1.0, 1.0))
    shape = (pages, case["Hkv"], case["page"], case["D"])
    shape = shape if layers is None else (layers,) + shape
    return dict(k_cache=_normal(shape, dtype, gen, 1.0 / k_scale),
                v_cache=_normal(shape, dtype, gen, 1.0 / v_scale), k_scale=k_scale, v_scale=v_scale)


def _prepare_batch(case, gen):
    """The packed batch: lengths, trees, the paged cache and its block table."""
    ctx, rows = _lengths(case)
    page, B = case["page"], case["B"]
    need = [-(-(c + n) // page) for c, n in zip(ctx, rows)]
    # where the context is not read, what precedes a request's last pages is a shared prefix
    shared = [0] * B if case["op"] == "attend" else [c // page for c in ctx]
    prefix = max(shared)
    own_pages = [n - s for n, s in zip(need, shared)]
    pages = prefix + sum(own_pages) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    at = torch.full((B, max(need) + 2), -1, dtype=torch.int64)
    used = prefix
    for b in range(B):
        at[b, :shared[b]] = torch.arange(shared[b])
        at[b, shared[b]:need[b]] = torch.arange(used, used + own_pages[b])
        used += own_pages[b]
    at = at.to(DEV)
    table = torch.where(at >= 0, order[at.clamp(min=0)], torch.full_like(at, -1, dtype=torch.int32))
    capacity = B * _max_rows(case)
    s = dict(op=case["op"], cu=_cu(rows), ctx=_ints(ctx), table=table.contiguous(),
             max_rows=_max_rows(case), longest=max(c + n for c, n in zip(ctx, rows)),
             capacity=capacity, window=case["window"], sinks=case["sinks"], deepest=case["depth"],
             total=sum(rows))
    s.update(_pools(case, pages, gen, case.get("layers")))
    if case["rows"] == "tree":
        trees = _trees(case, rows)
        flat = lambda i: sum((t[i] for t in trees), [])  # noqa: E731
        fill = [0] * (capacity - sum(rows))
        s["parents"] = _ints(flat(0) + fill)
        s["depths"] = _ints(flat(1) + fill)
    return s


def _prepare_enter(case, gen):
    s = _prepare_batch(case, gen)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    # queries, keys and values as the fused projection leaves them: one row per token
    s["qkv"] = _normal((s["capacity"], (Hq + 2 * Hkv) * D), torch.bfloat16, gen)
    half = case["rot"] // 2
    angle = (torch.arange(s["longest"], dtype=torch.float64, device=DEV)[:, None]
             * 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half))
    s.update(Hq=Hq, Hkv=Hkv, D=D, cos=angle.cos().float(), sin=angle.sin().float(),
             interleaved=case["interleaved"],
             depths=torch.zeros(s["capacity"], dtype=torch.int32, device=DEV),
             masks=torch.zeros((s["capacity"], -(-s["max_rows"] // 32)), dtype=torch.int32, device=DEV),
             out=torch.zeros((s["capacity"], Hq, D), dtype=torch.bfloat16, device=DEV))
    return s


def _prepare_attend(case, gen):
    s = _prepare_batch(case, gen)
    shape = (s["capacity"], case["Hq"], case["D"])
    s.update(q=_normal(shape, torch.bfloat16, gen, 1.5),
             out=torch.zeros(shape, dtype=torch.bfloat16, device=DEV), masks=None)
    if case["rows"] == "tree":  # made once per step, for all layers of one window
        s["masks"] = _packed_masks(s)[1]
    else:
        s["depths"] = None
    return s


def _prepare_commit(case, gen):
    """The target's choices follow some branch of every tree for a while."""
    s = _prepare_batch(case, gen)
    _, rows = _lengths(case)
    rng = random.Random(case["mix"] + 2)
    tokens = torch.randint(0, 150000, (s["capacity"],), generator=gen, device=DEV).to(torch.int32)
    choice = torch.randint(0, 150000, (s["capacity"],), generator=gen, device=DEV).to(torch.int32)
    steps, start = [], 0
    for n, (parents, depth) in zip(rows, _trees(case, rows)):
        # a branch outside the likeliest chain mostly, and that chain or a part of it else;
        # the first nodes are that chain, so no node of a branch lies where another one goes
        leaf = rng.randrange(n) if rng.random() < 0.8 else min(rng.randint(0, case["depth"]), n - 1)
        while leaf > 0:
            steps.append((start + parents[leaf], start + leaf))
            leaf = parents[leaf]
        start += n
    if steps:
        at = torch.tensor(steps, dtype=torch.int64, device=DEV)
        choice[at[:, 0]] = tokens[at[:, 1]]
    s.update(tokens=tokens, choice=choice, width=min(case["depth"] + 1, s["max_rows"]))
    return s


def _prepare_fork(case, gen):
    """Rows of B prompts and, behind them, of the answers that share their pages."""
    ctx, _ = _lengths(case)
    B, n, page = case["B"], case["copies"] - 1, case["page"]
    R = B * (n + 1)
    src = [i // n for i in range(B * n)]
    held = [-(-c // page) for c in ctx]
    grown = [-(-(c + 1) // page) for c in ctx]
    pages = sum(held) + B + 2 * n * B + 7  # a page to copy into and one to grow by for every row
    order = torch.randperm(sum(held), generator=gen, device=DEV).to(torch.int32)
    table = torch.full((R, max(grown) + 1), -1, dtype=torch.int32, device=DEV)
    used = 0
    for b in range(B):
        table[b, :held[b]] = order[used:used + held[b]]
        used += held[b]
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[:used] = 1
    s = dict(op="fork", table=table, held=_ints(held + [0] * (R - B)), refs=refs, page=page,
             before=_ints(ctx + [0] * (R - B)), lens=_ints(ctx + [0] * (R - B)),
             after=_ints([c + 1 for c in ctx] + [ctx[p] + 1 for p in src]), src=_ints(src),
             dst=_ints(list(range(B, R))))
    s.update(_pools(case, pages, gen, case["layers"]))
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + case["mix"])
    return {"enter": _prepare_enter, "attend": _prepare_attend, "commit": _prepare_commit,
            "fork": _prepare_fork}[case["op"]](case, gen)


# ------------------------------------------------------------------- the work

def _paths(case, rows):
    """Nodes that move in a commit, at most: those of every request's planted branch."""
    rng = random.Random(case["mix"] + 2)
    moved = 0
    for n, (parents, depth) in zip(rows, _trees(case, rows)):
        leaf = rng.randrange(n) if rng.random() < 0.8 else min(rng.randint(0, case["depth"]), n - 1)
        while leaf > 0:
            moved += leaf != depth[leaf]
            leaf = parents[leaf]
    return moved


def work(case):
    ctx, rows = _lengths(case)
    total, B = sum(rows), case["B"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    item = 1 if case["cache"] == "e4m3" else 2
    words = -(-_max_rows(case) // 32)
    slot = 2 * Hkv * D * item  # keys and values of a position
    if case["op"] == "enter":
        moved = total * ((2 * Hq + 2 * Hkv) * D * 2 + slot + case["rot"] * 4 + 4 * words + 12)
        return {"bytes": moved, "flops": total * (Hq + Hkv) * case["rot"] * 3}
    if case["op"] == "commit":
        moved = _paths(case, rows)
        return {"bytes": moved * slot * case["layers"] * 2 + total * 12 + B * (4 * case["depth"] + 20),
                "flops": total}
    if case["op"] == "fork":
        n = case["copies"] - 1
        slots = sum(c % page for c in ctx) * n
        entries = sum(-(-c // page) for c in ctx) * n
        return {"bytes": slots * slot * case["layers"] * 2 + entries * 12 + B * (n + 1) * 24,
                "flops": entries}
    window, sinks = case["window"] or 1 << 40, case["sinks"]
    tree = case["rows"] == "tree"
    depths = [t[1] for t in _trees(case, rows)] if tree else None
    kept = pairs = 0
    for b, (c, n) in enumerate(zip(ctx, rows)):
        low = max(0, c + 1 - window)  # positions that only sinks keep below it
        kept += c + n - low + min(low, sinks)
        for j in range(n):
            p = c + (depths[b][j] if tree else j)
            gone = max(0, p + 1 - window)
            pairs += p + 1 - gone + min(gone, sinks)
    return {"bytes": kept * slot + 2 * total * Hq * D * 2 + total * (4 + 4 * words if tree else 0)
            + sum(-(-(c + n) // page) for c, n in zip(ctx, rows)) * 4,
            "flops": pairs * Hq * D * 4}


# ------------------------------------------------------------ the plain forms

def _rows_of(s):
    """(row, request, place among its rows, whether it is a row) of every packed row."""
    live = torch.arange(s["capacity"], device=DEV) < s["cu"][-1]
    r = torch.minimum(torch.arange(s["capacity"], device=DEV), s["cu"][-1] - 1).long()
    b = torch.searchsorted(s["cu"], r.to(torch.int32), right=True) - 1
    return r, b, r - s["cu"].long()[b], live


def _seen_rows(s):
    """(depths, [row, node of its request] booleans): the ancestors in the window or the sinks."""
    _, b, j, live = _rows_of(s)
    start, ctx = s["cu"].long()[b], s["ctx"].long()[b]
    parents, W = s["parents"].long(), s["max_rows"]
    up = [torch.where(live, j, torch.full_like(j, -1))]  # the node, its parent, and so on
    for _ in range(s["deepest"]):
        k = up[-1]
        up.append(torch.where(k > 0, parents[start + k.clamp(min=0)], torch.full_like(k, -1)))
    depth = sum((k >= 0).long() for k in up) - 1
    seen = torch.zeros((s["capacity"], W), dtype=torch.bool, device=DEV)
    for step, k in enumerate(up):
        see = k >= 0
        if s["window"] and step >= s["window"]:
            see &= ctx + depth - step < s["sinks"]
        seen |= see[:, None] & (torch.arange(W, device=DEV) == k[:, None])
    return depth, seen


def _packed_masks(s):
    depth, seen = _seen_rows(s)
    words = -(-s["max_rows"] // 32)
    seen = torch.nn.functional.pad(seen, (0, 32 * words - s["max_rows"]))
    bit = torch.ones((), dtype=torch.int64, device=DEV) << torch.arange(32, device=DEV)
    masks = (seen.view(-1, words, 32) * bit).sum(-1)
    return depth, torch.where(masks >= 1 << 31, masks - (1 << 32), masks).to(torch.int32)


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    part, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([part, rest], -1)


def _raw(cache):
    return cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache


def _stored(x, scale, dtype):
    if dtype == torch.float8_e4m3fn:
        return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(dtype).view(torch.uint8)
    return x.to(dtype)


def _plain_enter(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    r, b, j, live = _rows_of(s)
    depth, masks = _packed_masks(s)
    s["depths"].copy_(torch.where(live, depth, s["depths"].long()))
    s["masks"].copy_(torch.where(live[:, None], masks, s["masks"]))
    x = s["qkv"][r].float()
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:]
    place, pos = s["ctx"].long()[b] + j, s["ctx"].long()[b] + depth[r]
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _rotate(q.view(-1, Hq, D), cos, sin, s["interleaved"]).to(torch.bfloat16)
    k = _rotate(k.reshape(-1, Hkv, D), cos, sin, s["interleaved"])
    page = s["k_cache"].shape[2]
    at, off = s["table"][b, place // page].long(), place % page
    _raw(s["k_cache"])[at, :, off] = _stored(k, s["k_scale"], s["k_cache"].dtype)
    _raw(s["v_cache"])[at, :, off] = _stored(v.reshape(-1, Hkv, D), s["v_scale"], s["v_cache"].dtype)
    s["out"].copy_(torch.where(live[:, None, None], q, s["out"]))
    return s["depths"], s["masks"], s["out"], s["k_cache"], s["v_cache"]


def _gathered(cache, table, pos):
    """The cache's rows at `pos` of every request, [B, Hkv, len, D] in 32 bits."""
    page = cache.shape[2]
    x = _raw(cache)[table[:, pos // page].long().clamp(min=0), :, (pos % page).expand(table.shape[0], -1)]
    return x.view(cache.dtype).float().transpose(1, 2)


def _plain_attend(s):
    q, cu, ctx = s["q"], s["cu"].long(), s["ctx"].long()
    Hq, D, Hkv, W = q.shape[1], q.shape[2], s["k_cache"].shape[1], s["max_rows"]
    B, G = ctx.numel(), Hq // Hkv
    j = torch.arange(W, device=DEV)
    row = (cu[:-1, None] + j).clamp(max=q.shape[0] - 1)
    t = torch.arange(s["longest"], device=DEV)
    wide = q[row].float().view(B, W, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * G, D)
    k = _gathered(s["k_cache"], s["table"], t)
    score = torch.matmul(wide, k.transpose(2, 3)).mul_(s["k_scale"] / math.sqrt(D))
    at = ctx[:, None] + (s["depths"].long()[row] if s["masks"] is not None else j)
    seen = torch.ones((), dtype=torch.bool, device=DEV)
    if s["window"]:
        seen = (t > at[:, :, None] - s["window"]) | (t < s["sinks"])
    if s["masks"] is not None:
        node = (t - ctx[:, None])[:, None].expand(B, W, -1)  # which new row a position holds
        inside = (node >= 0) & (node < W)
        word = s["masks"].long()[row].gather(2, node.clamp(0, W - 1) // 32)
        seen = torch.where(node < 0, seen, inside & ((word >> (node.clamp(0, W - 1) % 32)) & 1 > 0))
    else:
        seen = seen & (t <= at[:, :, None])
    score = score.view(B, Hkv, W, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    # rows past a request's own may see nothing; they are dropped below
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["table"], t)
    o = torch.matmul(p.view(B, Hkv, W * G, -1), v).view(B, Hkv, W, G, D).mul_(s["v_scale"]) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(B, W, Hq, D)
    _, b, place, live = _rows_of(s)
    s["out"].copy_(torch.where(live[:, None, None], o[b, place].to(q.dtype), s["out"]))
    return s["out"]


def _plain_commit(s):
    cu, parents, W = s["cu"].long(), s["parents"], s["max_rows"]
    B, layers = cu.numel() - 1, s["k_cache"].shape[0]
    j = torch.arange(W, device=DEV)
    row = (cu[:-1, None] + j).clamp(max=parents.numel() - 1)
    mine = j < (cu[1:] - cu[:-1])[:, None]
    parent, token, choice = parents[row].long(), s["tokens"][row], s["choice"][row]
    cur = torch.zeros(B, dtype=torch.int64, device=DEV)
    walking = torch.ones(B, dtype=torch.bool, device=DEV)
    path = [cur.clone()]
    for _ in range(s["width"] - 1):
        want = choice.gather(1, cur[:, None])
        child = mine & (j > cur[:, None]) & (parent == cur[:, None]) & (token == want)
        at = torch.where(child, j, W).amin(1)
        walking = walking & (at < W)
        cur = torch.where(walking, at, cur)
        path.append(torch.where(walking, at, -1))
    path = torch.stack(path, 1)
    accepted = (path >= 0).sum(1) - 1
    bonus = choice.gather(1, cur[:, None])[:, 0]
    page, ctx = s["k_cache"].shape[3], s["ctx"].long()[:, None]
    moves = path > 0
    b, i = moves.nonzero(as_tuple=True)
    old, new = (ctx + path)[b, i], (ctx + torch.arange(s["width"], device=DEV))[b, i]
    old = (s["table"][b, old // page].long(), old % page)
    new = (s["table"][b, new // page].long(), new % page)
    for cache in (_raw(s["k_cache"]), _raw(s["v_cache"])):
        for layer in range(layers):
            cache[layer][new[0], :, new[1]] = cache[layer][old[0], :, old[1]]
    return accepted.to(torch.int32), bonus, path.to(torch.int32), s["k_cache"], s["v_cache"]


def _plain_resize(s, lens):
    table, held, refs = s["table"], s["held"], s["refs"]
    want = -(-lens // s["page"])
    e = torch.arange(table.shape[1], device=DEV)
    gone = (e >= want[:, None]) & (e < held[:, None])
    pages = table[gone].long()
    refs.index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    table.masked_fill_(gone, -1)
    need = (want - held).clamp(min=0)
    before = need.cumsum(0) - need
    free = torch.argsort((refs > 0).to(torch.int32), stable=True).to(torch.int32)
    fresh = (e >= held[:, None]) & (e < want[:, None])
    taken = free[(before[:, None] + e - held[:, None])[fresh]]
    table[fresh] = taken
    refs[taken.long()] = 1
    held.copy_(want)


def _plain_fork(s):
    table, held, refs, page = s["table"], s["held"], s["refs"], s["page"]
    _plain_resize(s, s["before"])
    src, dst = s["src"].long(), s["dst"].long()
    full, rest = s["lens"][src] // page, s["lens"][src] % page
    e = torch.arange(table.shape[1], device=DEV)
    kept = e < full[:, None]
    rows = torch.where(kept, table[src], -1)
    pages = rows[kept].long()
    refs.index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    part = rest > 0
    free = torch.argsort((refs > 0).to(torch.int32), stable=True).to(torch.int32)
    fresh = free[(part.long().cumsum(0) - 1).clamp(min=0)]
    copy_src = torch.where(part, table[src].gather(1, full.long()[:, None])[:, 0], -1)
    copy_dst = torch.where(part, fresh, -1)
    rows = torch.where((e == full[:, None]) & part[:, None], fresh[:, None], rows)
    refs[fresh[part].long()] = 1
    table[dst] = rows
    held[dst] = full + part.to(torch.int32)
    off = torch.arange(page, device=DEV)
    which, slot = ((off < rest[:, None]) & part[:, None]).nonzero(as_tuple=True)
    for cache in (_raw(s["k_cache"]), _raw(s["v_cache"])):
        for layer in range(cache.shape[0]):
            cache[layer][copy_dst[which].long(), :, slot] = cache[layer][copy_src[which].long(), :, slot]
    _plain_resize(s, s["after"])
    return (table, held, refs, copy_src, copy_dst, torch.where(part, rest, 0), s["k_cache"],
            s["v_cache"])


def _own_enter(dspark, s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    depths, masks = dspark.dspark_tree_masks(
        s["parents"], s["cu"], s["max_rows"], ctx_lens=s["ctx"], window=s["window"],
        sinks=s["sinks"], out=(s["depths"], s["masks"]))
    q, k, v = s["qkv"].view(-1, Hq + 2 * Hkv, D).split((Hq, Hkv, Hkv), 1)
    q = dspark.dspark_append_tree_kv(
        q, k, v, s["cos"], s["sin"], depths, s["cu"], s["ctx"], s["table"], s["k_cache"],
        s["v_cache"], interleaved=s["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"],
        out=s["out"])
    return depths, masks, q, s["k_cache"], s["v_cache"]


def _own_attend(dspark, s):
    return dspark.dspark_tree_attention(
        s["q"], s["k_cache"], s["v_cache"], s["cu"], s["ctx"], s["table"], s["max_rows"],
        depths=s["depths"], masks=s["masks"], window=s["window"], sinks=s["sinks"],
        k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])


def _own_commit(dspark, s):
    accepted, bonus, path = dspark.dspark_tree_accept(
        s["choice"], s["tokens"], s["parents"], s["cu"], s["max_rows"], s["width"])
    dspark.dspark_move_kv(s["k_cache"], s["v_cache"], path, accepted, s["ctx"], s["table"])
    return accepted, bonus, path, s["k_cache"], s["v_cache"]


def _own_fork(dspark, s):
    pool = (s["table"], s["held"], s["refs"])
    dspark.dspark_resize_pages(*pool, s["before"], s["page"])
    copy_src, copy_dst, slots, _ = dspark.dspark_fork_pages(*pool, s["src"], s["dst"], s["lens"],
                                                           s["page"])
    dspark.dspark_copy_pages(s["k_cache"], s["v_cache"], copy_src, copy_dst, slots)
    dspark.dspark_resize_pages(*pool, s["after"], s["page"])
    return (s["table"], s["held"], s["refs"], copy_src, copy_dst, slots, s["k_cache"], s["v_cache"])


def run(state):
    if own:
        import confidence_scheduled_ragged_amd as dspark
        return {"enter": _own_enter, "attend": _own_attend, "commit": _own_commit,
                "fork": _own_fork}[state["op"]](dspark, state)
    return {"enter": _plain_enter, "attend": _plain_attend, "commit": _plain_commit,
            "fork": _plain_fork}[state["op"]](state)


# --------------------------------------------------- the definitions, 64 bits

def _exact_enter(case, s):
    ctx, rows = _lengths(case)
    Hq, Hkv, D, page, half = s["Hq"], s["Hkv"], s["D"], case["page"], case["rot"] // 2
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    out, depths, masks = s["out"].double(), s["depths"].tolist(), s["masks"].tolist()
    pairs = [(2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half) for i in range(half)]
    first, second = (torch.tensor(p, device=DEV) for p in zip(*pairs))
    limit = E4M3_MAX if case["cache"] == "e4m3" else math.inf
    parents, start = s["parents"].tolist(), 0
    for b in range(case["B"]):
        n, line = rows[b], []
        for j in range(n):
            up, k = [j], parents[start + j]
            while k >= 0:
                up.append(k)
                k = parents[start + k]
            depth = len(up) - 1
            line.append(ctx[b] + depth)
            depths[start + j] = depth
            word = [0] * len(masks[0])
            for step, k in enumerate(up):
                if not case["window"] or step < case["window"] or ctx[b] + depth - step < case["sinks"]:
                    word[k // 32] += 1 << (k % 32)
            masks[start + j] = [w - (1 << 32) if w >> 31 else w for w in word]
        x = s["qkv"][start:start + n].double().view(n, Hq + 2 * Hkv, D)
        pos = torch.tensor(line, device=DEV)
        turn = torch.complex(s["cos"].double()[pos], s["sin"].double()[pos])[:, None]
        z = torch.complex(x[:, :Hq + Hkv, first], x[:, :Hq + Hkv, second]) * turn
        y = x.clone()
        y[:, :Hq + Hkv, first], y[:, :Hq + Hkv, second] = z.real, z.imag
        out[start:start + n] = y[:, :Hq]
        place = torch.arange(ctx[b], ctx[b] + n, device=DEV)
        at, off = s["table"][b].long()[place // page], place % page
        k_cache[at, :, off] = (y[:, Hq:Hq + Hkv] / s["k_scale"]).clamp(-limit, limit)
        v_cache[at, :, off] = (y[:, Hq + Hkv:] / s["v_scale"]).clamp(-limit, limit)
        start += n
    return _ints(depths), _ints(masks), out, k_cache, v_cache


def _exact_attend(case, s):
    """Request by request: every head's scores, their softmax over what a row sees, the mean."""
    ctx, rows = _lengths(case)
    page, D, Hkv, window, sinks = case["page"], case["D"], case["Hkv"], case["window"], case["sinks"]
    trees = _trees(case, rows) if case["rows"] == "tree" else None
    out = s["out"].double()
    start = 0
    for b in range(case["B"]):
        c, n = ctx[b], rows[b]
        low = max(0, c + 1 - window) if window else 0
        t = torch.cat([torch.arange(min(low, sinks)), torch.arange(low, c + n)]).to(DEV)
        pages = s["table"][b].long()[t // page]
        k = s["k_cache"][pages, :, t % page].double() * s["k_scale"]
        v = s["v_cache"][pages, :, t % page].double() * s["v_scale"]
        # positions of what is cached and of the rows, and which rows are ancestors of which
        depth = torch.tensor(trees[b][1] if trees else range(n), device=DEV)
        where = torch.where(t < c, t, c + depth[(t - c).clamp(min=0)])
        family = torch.zeros((n, n), dtype=torch.bool)
        for j in range(n):
            if trees:
                a = j
                while a >= 0:
                    family[j, a] = True
                    a = trees[b][0][a]
            else:
                family[j, :j + 1] = True
        hidden = torch.zeros((n, t.numel()), dtype=torch.bool, device=DEV)
        hidden[:, t.numel() - n:] = ~family.to(DEV)
        if window:
            hidden |= ((c + depth)[:, None] - where >= window) & (where >= sinks)
        q = s["q"][start:start + n].double().view(n, Hkv, -1, D)
        for h in range(Hkv):
            score = torch.tensordot(q[:, h], k[:, h], dims=([2], [1])) / math.sqrt(D)
            share = score.masked_fill(hidden[:, None], -math.inf).softmax(2)
            out[start:start + n].view(n, Hkv, -1, D)[:, h] = torch.tensordot(
                share, v[:, h], dims=([2], [0]))
        start += n
    return out


def _exact_commit(case, s):
    ctx, rows = _lengths(case)
    parents, tokens, choice = (s[k].tolist() for k in ("parents", "tokens", "choice"))
    table, page = s["table"].tolist(), case["page"]
    accepted, bonus, paths, old, new = [], [], [], [], []
    start = 0
    for b in range(case["B"]):
        path = [0]
        while len(path) < s["width"]:
            here = path[-1]
            child = [j for j in range(here + 1, rows[b])
                     if parents[start + j] == here and tokens[start + j] == choice[start + here]]
            if not child:
                break
            path.append(child[0])
        for i, j in enumerate(path[1:], 1):
            a, z = ctx[b] + j, ctx[b] + i
            old.append((table[b][a // page], a % page))
            new.append((table[b][z // page], z % page))
        accepted.append(len(path) - 1)
        bonus.append(choice[start + path[-1]])
        paths.append(path + [-1] * (s["width"] - len(path)))
        start += rows[b]
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    if old:
        (a, i), (z, j) = (torch.tensor(p, device=DEV).t() for p in (old, new))
        for layer in range(case["layers"]):
            for c in (k_cache[layer], v_cache[layer]):
                c[z, :, j] = c[a, :, i]
    return _ints(accepted), _ints(bonus), _ints(paths), k_cache, v_cache


def _exact_fork(case, s):
    """One page after the other, on the host: the lowest free page is always the next."""
    page = case["page"]
    table, held, refs = s["table"].tolist(), s["held"].tolist(), s["refs"].tolist()

    def fresh(b):
        p = refs.index(0)
        refs[p] = 1
        table[b][held[b]] = p
        held[b] += 1
        return p

    def resize(lens):
        want = [-(-n // page) for n in lens.tolist()]
        for b, w in enumerate(want):
            while held[b] > w:
                held[b] -= 1
                refs[table[b][held[b]]] -= 1
                table[b][held[b]] = -1
        for b, w in enumerate(want):
            while held[b] < w:
                fresh(b)

    resize(s["before"])
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    copies = []
    for a, z in zip(s["src"].tolist(), s["dst"].tolist()):
        full, rest = divmod(int(s["lens"][a]), page)
        for e in range(full):
            table[z][e] = table[a][e]
            refs[table[a][e]] += 1
        held[z] = full
        copies.append((table[a][full], fresh(z), rest) if rest else (-1, -1, 0))
    for a, z, rest in copies:
        if rest:
            for c in (k_cache, v_cache):
                c[:, z, :, :rest] = c[:, a, :, :rest]
    resize(s["after"])
    return (_ints(table), _ints(held), _ints(refs), *(_ints(x) for x in zip(*copies)), k_cache,
            v_cache)


def exact(case, seed):
    s = prepare(case, seed)
    return {"enter": _exact_enter, "attend": _exact_attend, "commit": _exact_commit,
            "fork": _exact_fork}[case["op"]](case, s)
