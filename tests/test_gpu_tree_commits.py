"""The loop of examples/tree_loop.py (needs an MI355X) where the target's choices are
planted, so that nodes beside the first chain are accepted: their keys and values have
to be moved, and later steps read them. And the choices of trees that have more rows
than a block of dspark_accept."""
import random

import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
import tree_ref as ref
from test_gpu_tree import forest, i32, starts
from test_gpu_tree_loop import PROMPTS, example

pytestmark = pytest.mark.gpu

DEV = "cuda:0"

# ways from the root to a leaf of the example's tree, three of them beside its first chain
WAYS = ([0, 4, 7, 8], [0, 1, 6, 9], [0, 5], [0, 1, 2, 3])


class Planted(example.Target):
    """Puts the choices of a way down every tree into the logits; `clean` is without them."""

    ways = None

    def forward(self, tokens, cu, ctx, table, max_rows, parents=None):
        self.clean = super().forward(tokens, cu, ctx, table, max_rows, parents)
        if parents is None or self.ways is None:
            return self.clean
        logits, n, line = self.clean.clone(), len(example.TREE), tokens.tolist()
        for b, way in enumerate(self.ways):
            for up, down in zip(way, way[1:]):
                logits[b * n + up, line[b * n + down]] += 1000
        return logits


def plain_logits(t, seq):
    """The last token's logits over one sequence in 32 bits, keys and values rounded as
    the cache holds them."""
    x = t.embed[torch.tensor(seq, device=t.device)].float()
    n, G, half = len(seq), t.Hq // t.Hkv, t.D // 2
    cos, sin = t.cos[:n, None], t.sin[:n, None]
    at = torch.arange(n, device=t.device)

    def turn(y):
        a, b = y[..., :half], y[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    def norm(y):
        return y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)

    def cached(y):
        limit = torch.finfo(t.k.dtype).max
        return (y / t.scale).clamp(-limit, limit).to(t.k.dtype).float() * t.scale
    for w, view in zip(t.layers, t.views):
        hidden = at > at[:, None]
        if view["window"]:
            hidden = hidden | ((at[:, None] - at >= view["window"]) & (at >= view["sinks"]))
        y = (norm(x) @ w["qkv"].float().t()).view(n, t.Hq + 2 * t.Hkv, t.D)
        q, k, v = y.split((t.Hq, t.Hkv, t.Hkv), 1)
        q, k, v = turn(q), cached(turn(k)), cached(v)
        o = torch.empty_like(q)
        for h in range(t.Hq):
            s = (q[:, h] @ k[:, h // G].t().contiguous()) * t.D ** -0.5
            o[:, h] = s.masked_fill(hidden, float("-inf")).softmax(-1) @ v[:, h // G].contiguous()
        x = x + o.flatten(1) @ w["o"].float().t()
        x = x + torch.relu(norm(x) @ w["up"].float().t()) @ w["down"].float().t()
    return (norm(x) @ t.head.float().t())[-1]


def apart(a, b):
    return float((a.float() - b).square().mean().sqrt() / b.square().mean().sqrt())


@pytest.mark.parametrize("cache,bound", [(torch.bfloat16, 0.015), (torch.float8_e4m3fn, 0.025)])
def test_accepted_branches_are_moved_and_read(cache, bound):
    """Some twenty bf16 roundings on the way to the logits, nine a layer and two after
    them, each off by 2^-7 / 12^.5 in the mean square of values from 1 to 2, 1.7e-3 of
    the values: 20^.5 * 1.7e-3 = 0.008 if each came through whole, bounded by twice that.
    With 8 bits the keys and values that lie within a bf16 rounding (2^-8 of 2^-3 to 2^-4
    a step, about one in 16) of a border fall on its other side: 16^-.5 * 0.09 = 0.022 of
    the attention's result, which is less than a third of what it is added to: 0.008, in
    two layers 0.011, and 0.014 together with the roundings.
    What a cache without the moves would answer is off by more than that."""
    t = Planted(cache=cache)
    loop = example.Loop(t, PROMPTS, answers=3)
    seqs = [list(PROMPTS[b % 3]) for b in range(loop.B)]
    unmoved = [list(s) for s in seqs]
    rng, moved, seen_apart = random.Random(7), 0, 0.0
    for turn in range(6):
        t.ways = [WAYS[(turn + b) % 4] if turn % 2 else rng.choice(WAYS) for b in range(loop.B)]
        loop.new_numbers()
        tokens, accepted, bonus, path, _ = loop.step()
        tokens, path, n = tokens.tolist(), path.tolist(), loop.n
        for b, (seq, way) in enumerate(zip(seqs, t.ways)):
            for j in (0, 3, 8, 9):  # the root and leaves see all that is committed
                line, k = [], j
                while k >= 0:
                    line.append(tokens[b][k])
                    k = example.TREE[k][0]
                want = plain_logits(t, seq + line[::-1])
                err = apart(t.clean[b * n + j], want)
                assert err < bound, (turn, b, j, err)
                if j == 0 and unmoved[b] != seq:
                    seen_apart = max(seen_apart, apart(plain_logits(t, unmoved[b] + line), want))
            a = int(accepted[b])
            assert path[b] == way + [-1] * (loop.width - len(way)) and a == len(way) - 1
            moved += sum(i != j for i, j in enumerate(way))
            seqs[b] = seq + [tokens[b][j] for j in way]
            unmoved[b] = seq + tokens[b][:a + 1]
            assert loop.root[b] == bonus[b]
        assert loop.ctx.tolist() == [len(s) for s in seqs]
    assert moved >= 60
    assert seen_apart > 4 * bound


@pytest.mark.parametrize("drawn", [False, True])
def test_choices_of_trees_of_more_rows_than_a_block(drawn):
    """A row's choice is its own: the packed rows of large trees go through dspark_accept
    and dspark_sample_accept as blocks of up to 257 rows."""
    rows, V, g1 = [600, 3, 257, 350], 40, 200
    cu, total = starts(rows), sum(rows)
    blocks = [0]
    while blocks[-1] < total:
        blocks.append(min(blocks[-1] + g1 - len(blocks) % 3, total))
    B = len(blocks) - 1
    gen = torch.Generator(device=DEV).manual_seed(3)
    logits = torch.randn((B * g1, V), generator=gen, device=DEV).bfloat16()
    blank = torch.zeros((B, g1), dtype=torch.int32, device=DEV)
    if drawn:
        top = torch.ones(B, dtype=torch.int32, device=DEV)
        numbers = torch.rand(B * g1, generator=gen, device=DEV)
        choice = dspark.dspark_sample_accept(logits, None, i32(blocks), blank, numbers, top_k=top)[0]
    else:
        choice = dspark.dspark_accept(logits, None, i32(blocks), blank)[0]
    # the lowest index of the largest logit
    want = [row.index(max(row)) for row in logits.float().tolist()]
    assert choice[:total].tolist() == want[:total]
    parents, tokens = forest(rows, 5), [0] * total
    rng = random.Random(2)
    for b, n in enumerate(rows):  # the target goes some way down every tree
        for j in range(1, n):
            up = cu[b] + parents[cu[b] + j]
            tokens[cu[b] + j] = want[up] if rng.random() < 0.7 else rng.randrange(V)
    got = dspark.dspark_tree_accept(choice[:total], i32(tokens), i32(parents), i32(cu), 600, 90)
    for g, w in zip(got, ref.accept(want, tokens, parents, cu, 600, 90)):
        assert g.tolist() == w
    assert max(got[0].tolist()) > 3
