"""The verify loop of examples/verify_loop.py (needs an MI355X): its logits
against a plain forward over each request's whole sequence, its commits against
the tokens drawn, and its captured step against the eager one."""
import importlib.util
import os

import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark  # noqa: F401

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "verify_loop.py")
spec = importlib.util.spec_from_file_location("verify_loop", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)

PROMPTS = [[5, 17, 300], list(range(40, 90)), [7] * 20, [999]]


def plain_logits(t, seq):
    """The target over one sequence in 32 bits, no cache and no kernels of ours."""
    x = t.embed[torch.tensor(seq, device=t.device)].float()
    n, G, half = len(seq), t.Hq // t.Hkv, t.D // 2
    cos, sin = t.cos[:n, None], t.sin[:n, None]

    def turn(y):
        a, b = y[..., :half], y[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    hidden = torch.ones((n, n), dtype=torch.bool, device=t.device).triu(1)

    def norm(y):
        return y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
    for w in t.layers:
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
    return norm(x) @ t.head.float().t()


@pytest.mark.parametrize("cache,bound", [(torch.bfloat16, 0.15), (torch.float8_e4m3fn, 0.6)])
def test_logits_follow_the_plain_forward(cache, bound):
    """Logits spread by about 6; a residual of two layers carries some ten bf16
    roundings of 2^-8 (or 2^-4 of every cached value, averaged over the keys)."""
    t = example.Target(cache=cache)
    loop = example.Loop(t, PROMPTS)
    seqs = [list(p) for p in PROMPTS]
    accepted_any = 0
    for _ in range(6):
        loop.new_numbers()
        roots = loop.root.tolist()
        tokens, lengths, accepted, bonus, logits, cu = loop.step()
        tokens, lengths, cu = tokens.tolist(), lengths.tolist(), cu.tolist()
        for b in range(len(seqs)):
            assert tokens[b][0] == roots[b]
            window = tokens[b][:lengths[b] + 1]
            want = plain_logits(t, seqs[b] + window)[len(seqs[b]):]
            got = logits[cu[b]:cu[b + 1]].float()
            assert got.shape == want.shape
            err = (got - want).square().mean().sqrt() / want.square().mean().sqrt()
            assert float(err) < bound, (b, float(err))
            n = int(accepted[b])
            accepted_any += n
            seqs[b] += tokens[b][:n + 1]
            assert loop.root[b] == bonus[b]
        assert loop.ctx.tolist() == [len(s) for s in seqs]
    assert accepted_any > 0


def test_captured_steps_equal_eager_ones():
    eager = example.Loop(example.Target(), PROMPTS)
    other = example.Loop(example.Target(), PROMPTS)
    assert torch.equal(eager.root, other.root)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep = [x.clone() for x in (other.ctx, other.root)]
        other.step()
        other.ctx.copy_(keep[0])
        other.root.copy_(keep[1])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = other.step()
    for _ in range(6):
        eager.new_numbers()
        other.uniforms.copy_(eager.uniforms)
        want = [x.clone() for x in eager.step()[:4]]
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(held[:4], want):
            assert torch.equal(g, w)
        assert torch.equal(other.ctx, eager.ctx)
