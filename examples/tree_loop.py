"""Several answers to every prompt, drafted as trees, every step on the GPU.

Prompts enter a paged cache (dspark_resize_pages gives their rows pages); each is
answered several times by rows that share its pages (dspark_fork_pages and
dspark_copy_pages). A step drafts a tree of tokens per row, gives the rows pages for
it, runs the target over all nodes (dspark_tree_masks, then per layer
dspark_append_tree_kv and dspark_tree_attention; every other layer keeps a window and
the first positions), draws the target's tokens (dspark_sample_accept), walks down
the trees (dspark_tree_accept) and brings the accepted nodes together in the cache
(dspark_move_kv). Nothing is read back inside a step, so that it can be captured.

    python examples/tree_loop.py [--steps 16] [--answers 3] [--cache e4m3] [--graph]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import confidence_scheduled_ragged_amd as dspark  # noqa: E402
import verify_loop  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32

# parent and rank among its siblings of every node: the likeliest chain first
TREE = [(-1, 0), (0, 0), (1, 0), (2, 0), (0, 1), (0, 2), (1, 1), (4, 0), (7, 0), (6, 0)]


class Target(verify_loop.Target):
    """verify_loop's target with a window and sinks in every other layer."""

    def __init__(self, window=24, sinks=4, **kw):
        super().__init__(**kw)
        self.views = [dict(window=window if i % 2 else 0, sinks=sinks if i % 2 else 0)
                      for i in range(len(self.layers))]

    def forward(self, tokens, cu, ctx, table, max_rows, parents=None):
        """Logits of the packed rows: chains, or the nodes of trees (parents [rows])."""
        x = self.embed[tokens.clamp(min=0).long()]
        heads = (self.Hq, self.Hkv, self.Hkv)
        scales = dict(k_scale=self.scale, v_scale=self.scale)
        trees = {}
        if parents is not None:  # once per kind of layer
            for view in self.views[:2]:
                trees[view["window"]] = dspark.dspark_tree_masks(parents, cu, max_rows,
                                                                 ctx_lens=ctx, **view)
        for i, (w, view) in enumerate(zip(self.layers, self.views)):
            q, k, v = (self.norm(x) @ w["qkv"].t()).view(-1, sum(heads), self.D).split(heads, 1)
            pools = (self.k[i], self.v[i])
            depths, masks = trees.get(view["window"], (None, None))
            if parents is None:
                q = dspark.dspark_append_kv(q, k, v, self.cos, self.sin, cu, ctx, table, *pools,
                                            **scales)
            else:
                q = dspark.dspark_append_tree_kv(q, k, v, self.cos, self.sin, depths, cu, ctx, table,
                                                 *pools, **scales)
            o = torch.zeros_like(q)
            dspark.dspark_tree_attention(q, *pools, cu, ctx, table, max_rows, depths=depths,
                                         masks=masks, out=o, **view, **scales)
            x = x + o.flatten(1) @ w["o"].t()
            x = x + torch.relu(self.norm(x) @ w["up"].t()) @ w["down"].t()
        return self.norm(x) @ self.head.t()


class Loop:
    """`answers` rows per prompt: `step()` verifies one tree of drafts per row."""

    def __init__(self, target, prompts, answers=3, temperature=0.7, top_k=40, seed=1):
        t, dev, P = target, target.device, len(prompts)
        self.target, self.n, self.B = t, len(TREE), P * answers
        self.width = 1 + max(self._depth(j) for j in range(self.n))
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        pages = t.k.shape[1]
        self.pool = dspark.page_pool(pages, self.B, pages, dev)
        self.ctx = torch.zeros(self.B, dtype=I32, device=dev)
        f = lambda v: torch.full((self.B,), v, dtype=torch.float32, device=dev)  # noqa: E731
        self.sampling = dict(temperature=f(temperature),
                             top_k=torch.full((self.B,), top_k, dtype=I32, device=dev))
        # the drafter: the next tokens by the embedding alone
        ranks = 1 + max(rank for _, rank in TREE)
        self.next = (t.norm(t.embed) @ t.head.t()).topk(ranks, 1).indices.to(I32)
        self.parents = torch.tensor([p for p, _ in TREE] * self.B, dtype=I32, device=dev)
        self.cu = torch.arange(self.B + 1, dtype=I32, device=dev) * self.n
        self.tokens = torch.zeros((self.B, self.n), dtype=I32, device=dev)
        self.uniforms = torch.rand(self.B * self.n, generator=self.gen, device=dev)
        self.granted = torch.ones(self.B, dtype=I32, device=dev)
        self.root = self._prompts(prompts, answers)

    @staticmethod
    def _depth(j):
        return 0 if TREE[j][0] < 0 else 1 + Loop._depth(TREE[j][0])

    def _prompts(self, prompts, answers):
        """The prompts as packed chunks, then the forks; returns every row's first token."""
        t, dev, P = self.target, self.target.device, len(prompts)
        table, held, refs = self.pool
        lens = [len(p) for p in prompts]
        self.ctx[:P] = torch.tensor(lens, dtype=I32, device=dev)
        dspark.dspark_resize_pages(*self.pool, self.ctx, t.page, granted=self.granted)
        cu = torch.tensor([0] + lens, device=dev).cumsum(0).to(I32)
        tokens = torch.tensor([x for p in prompts for x in p], dtype=I32, device=dev)
        none = torch.zeros(P, dtype=I32, device=dev)
        logits = t.forward(tokens, cu, none, table[:P], max(lens))
        rows = torch.arange(self.B, dtype=I32, device=dev)
        if answers > 1:
            src, dst = rows[P:] % P, rows[P:].clone()
            *copies, granted = dspark.dspark_fork_pages(*self.pool, src, dst, self.ctx, t.page)
            dspark.dspark_copy_pages(t.k, t.v, *copies)
            self.granted[P:] = granted
            self.ctx[P:] = self.ctx[src.long()]
        # one row per answer in a block of as many as a tree has, nothing drafted
        last = logits[(cu[1:] - 1).long()][(rows % P).long()]
        block = last.repeat_interleave(self.n, 0)
        src = torch.full((self.B * self.n,), -1, dtype=I32, device=dev)
        src[:self.B] = rows * self.n
        ones = torch.arange(self.B + 1, dtype=I32, device=dev)
        _, _, bonus = dspark.dspark_sample_accept(block, src, ones, self.tokens, self.uniforms,
                                                  **self.sampling)
        return bonus.clone()

    def step(self):
        """Drafts, verifies and commits; returns (tokens, accepted, bonus, path, logits)."""
        t = self.target
        self.tokens[:, 0] = self.root
        for j, (p, rank) in enumerate(TREE[1:], 1):
            self.tokens[:, j] = self.next[self.tokens[:, p].long(), rank]
        granted = dspark.dspark_resize_pages(*self.pool, self.ctx + self.n, t.page)
        self.granted.mul_(granted)
        packed = self.tokens.view(-1)
        logits = t.forward(packed, self.cu, self.ctx, self.pool[0], self.n, self.parents)
        drawn, _, _ = dspark.dspark_sample_accept(logits, None, self.cu, self.tokens, self.uniforms,
                                                  **self.sampling)
        accepted, bonus, path = dspark.dspark_tree_accept(drawn, packed, self.parents, self.cu,
                                                          self.n, self.width)
        dspark.dspark_move_kv(t.k, t.v, path, accepted, self.ctx, self.pool[0])
        self.ctx += accepted + 1  # the root and the accepted drafts are in the cache
        self.root.copy_(bonus)
        return self.tokens, accepted, bonus, path, logits

    def new_numbers(self):
        self.uniforms.uniform_(generator=self.gen)


def captured(loop):
    """A step as a graph, its state put back to before it; returns (graph, its outputs)."""
    state = (loop.ctx, loop.root, loop.granted, *loop.pool)
    keep = [x.clone() for x in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # a step outside the graph allocates what steps share
        loop.step()
        for x, old in zip(state, keep):
            x.copy_(old)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = loop.step()
    return graph, held


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--answers", type=int, default=3)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--graph", action="store_true", help="capture a step and replay it")
    a = ap.parse_args()
    prompts, page = [[5, 17, 300], list(range(40, 90)), [7] * 20, [999]], 16
    longest = max(len(p) for p in prompts) + (a.steps + 1) * len(TREE)
    target = Target(cache=BF16 if a.cache == "bf16" else torch.float8_e4m3fn, page=page,
                    pages=len(prompts) * a.answers * -(-longest // page), longest=longest)
    loop = Loop(target, prompts, a.answers)
    out = [[t] for t in loop.root.tolist()]
    graph, held = captured(loop) if a.graph else (None, None)
    taken = 0
    for _ in range(a.steps):
        loop.new_numbers()
        if graph:
            graph.replay()
            tokens, accepted, bonus, path, _ = held
        else:
            tokens, accepted, bonus, path, _ = loop.step()
        rows = zip(tokens.tolist(), accepted.tolist(), bonus.tolist(), path.tolist())
        for b, (nodes, n, last, way) in enumerate(rows):
            out[b] += [nodes[j] for j in way[1:1 + n]] + [last]
            taken += n
    if not bool(loop.granted.all()):
        raise SystemExit("the cache has too few pages")
    for b, seq in enumerate(out):
        print(f"prompt {b % len(prompts)}, answer {b // len(prompts)}: {len(seq)} tokens, the first "
              f"{seq[:8]}")
    print(f"{a.steps} steps, {taken} drafts accepted, {int((loop.pool[2] > 1).sum())} pages shared")


if __name__ == "__main__":
    main()
