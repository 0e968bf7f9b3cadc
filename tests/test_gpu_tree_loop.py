"""The loop of examples/tree_loop.py (needs an MI355X): the logits of every node
against a plain forward over its whole sequence, commits against the tokens drawn,
pages against their counts, and the captured step against the eager one."""
import importlib.util
import os

import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark  # noqa: F401

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "tree_loop.py")
spec = importlib.util.spec_from_file_location("tree_loop", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)

PROMPTS = [[5, 17, 300], list(range(40, 90)), [999]]


def plain_logits(t, seq):
    """The last token's logits over one sequence in 32 bits, no cache and no kernels of ours."""
    x = t.embed[torch.tensor(seq, device=t.device)].float()
    n, G, half = len(seq), t.Hq // t.Hkv, t.D // 2
    cos, sin = t.cos[:n, None], t.sin[:n, None]
    at = torch.arange(n, device=t.device)

    def turn(y):
        a, b = y[..., :half], y[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    def norm(y):
        return y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
    for w, view in zip(t.layers, t.views):
        hidden = at > at[:, None]
        if view["window"]:
            hidden = hidden | ((at[:, None] - at >= view["window"]) & (at >= view["sinks"]))
        y = (norm(x) @ w["qkv"].float().t()).view(n, t.Hq + 2 * t.Hkv, t.D)
        q, k, v = y.split((t.Hq, t.Hkv, t.Hkv), 1)
        q, k = turn(q), turn(k).repeat_interleave(G, 1)
        v = v.repeat_interleave(G, 1)
        o = torch.empty_like(q)
        for h in range(t.Hq):
            s = (q[:, h] @ k[:, h].t().contiguous()) * t.D ** -0.5
            o[:, h] = s.masked_fill(hidden, float("-inf")).softmax(-1) @ v[:, h]
        x = x + o.flatten(1) @ w["o"].float().t()
        x = x + torch.relu(norm(x) @ w["up"].float().t()) @ w["down"].float().t()
    return (norm(x) @ t.head.float().t())[-1]


@pytest.mark.parametrize("cache,bound", [(torch.bfloat16, 0.15), (torch.float8_e4m3fn, 0.6)])
def test_every_nodes_logits_follow_the_plain_forward(cache, bound):
    """Logits spread by about 6; a residual of two layers carries some ten bf16
    roundings of 2^-8 (or 2^-4 of every cached value, averaged over the keys)."""
    t = example.Target(cache=cache)
    loop = example.Loop(t, PROMPTS, answers=3)
    seqs = [list(PROMPTS[b % 3]) for b in range(loop.B)]
    taken = 0
    for turn in range(5):
        loop.new_numbers()
        roots = loop.root.tolist()
        tokens, accepted, bonus, path, logits = loop.step()
        tokens, path, n = tokens.tolist(), path.tolist(), loop.n
        for b, seq in enumerate(seqs):
            assert tokens[b][0] == roots[b]
            for j in range(n):
                line, k = [], j
                while k >= 0:
                    line.append(tokens[b][k])
                    k = example.TREE[k][0]
                want = plain_logits(t, seq + line[::-1])
                got = logits[b * n + j].float()
                err = (got - want).square().mean().sqrt() / want.square().mean().sqrt()
                assert float(err) < bound, (turn, b, j, float(err))
            a = int(accepted[b])
            taken += a
            assert path[b][a + 1:] == [-1] * (loop.width - a - 1)
            for up, down in zip(path[b], path[b][1:a + 1]):
                assert example.TREE[down][0] == up
            seqs[b] = seq + [tokens[b][j] for j in path[b][:a + 1]]
            assert loop.root[b] == bonus[b]
        assert loop.ctx.tolist() == [len(s) for s in seqs]
    assert taken > 0
    # every entry of the table is one reference, and no page serves two rows' new positions
    table, held, refs = loop.pool
    named = table[table >= 0]
    assert torch.equal(torch.bincount(named, minlength=refs.numel()).int(), refs)
    assert held.tolist() == [-(-(len(s) - a + loop.n - 1) // t.page) for s, a in
                             zip(seqs, accepted.tolist())]
    assert bool(loop.granted.all())
    shared = {int(p) for p in (refs > 1).nonzero()}
    assert len(shared) == sum(len(p) // t.page for p in PROMPTS)


def test_captured_steps_equal_eager_ones():
    eager = example.Loop(example.Target(), PROMPTS)
    other = example.Loop(example.Target(), PROMPTS)
    assert torch.equal(eager.root, other.root)
    graph, held = example.captured(other)
    for _ in range(6):
        eager.new_numbers()
        other.uniforms.copy_(eager.uniforms)
        want = [x.clone() for x in eager.step()[:4]]
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(held[:4], want):
            assert torch.equal(g, w)
        for g, w in zip((other.ctx, *other.pool), (eager.ctx, *eager.pool)):
            assert torch.equal(g, w)


def test_rows_that_end_give_their_pages_back():
    loop = example.Loop(example.Target(), PROMPTS, answers=2)
    loop.step()
    loop.ctx[1] = 0
    keep = loop.ctx.clone()
    dspark.dspark_resize_pages(*loop.pool, keep, loop.target.page)
    table, held, refs = loop.pool
    assert int(held[1]) == 0 and bool((table[1] == -1).all())
    # the other answer to the same prompt still holds what they shared
    full = len(PROMPTS[1]) // loop.target.page
    assert refs[table[4, :full].long()].tolist() == [1] * full
    dspark.dspark_resize_pages(*loop.pool, torch.zeros_like(keep), loop.target.page)
    assert not bool(refs.any())


def test_the_example_runs(capsys, monkeypatch):
    for flags in ([], ["--graph", "--cache", "e4m3", "--answers", "1", "--steps", "3"]):
        monkeypatch.setattr("sys.argv", ["tree_loop.py", *flags])
        example.main()
        assert "drafts accepted" in capsys.readouterr().out
