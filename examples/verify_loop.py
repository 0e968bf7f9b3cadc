"""Speculative decoding with a small random target, every step on the GPU.

A step drafts gamma tokens per request, scores them (dspark_confidence), cuts
every request's window (dspark_schedule), packs the windows (dspark_compact),
runs the target over the packed rows (per layer dspark_append_kv and
dspark_verify_attention on a paged cache), draws the target's tokens and accepts
the drafts that agree (dspark_sample_accept). Prompts go through the same layers
as one chunk per request. Nothing is read back inside a step, so that a step can
be captured into a graph.

    python examples/verify_loop.py [--steps 32] [--cache e4m3] [--graph]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import confidence_scheduled_ragged_amd as dspark  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


class Target:
    """Random weights of a decoder with grouped heads, and its paged cache."""

    def __init__(self, layers=2, d=256, Hq=8, Hkv=2, D=64, V=1000, page=16, pages=512,
                 longest=1024, cache=BF16, device="cuda:0", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def w(*shape):
            x = torch.randn(shape, generator=gen, device=device)
            return (x * shape[-1] ** -0.5).to(BF16)
        self.Hq, self.Hkv, self.D, self.page, self.device = Hq, Hkv, D, page, device
        self.embed = (torch.randn((V, d), generator=gen, device=device) * 3).to(BF16)
        self.head = w(V, d) * 6  # logits spread by 6
        self.layers = [dict(qkv=w((Hq + 2 * Hkv) * D, d), o=w(d, Hq * D), up=w(2 * d, d),
                            down=w(d, 2 * d)) for _ in range(layers)]
        half = D // 2
        angle = (torch.arange(longest, dtype=torch.float64, device=device)[:, None]
                 * 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=device) / half))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        # an 8-bit cache holds values of about 1 times 1 / scale
        self.scale = 2.0 ** -6 if cache == torch.float8_e4m3fn else 1.0
        shape = (layers, pages, Hkv, page, D)
        self.k = torch.zeros(shape, dtype=BF16, device=device).to(cache)
        self.v = torch.zeros(shape, dtype=BF16, device=device).to(cache)

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).to(BF16)

    def forward(self, tokens, cu, ctx, table, max_rows):
        """Logits of the packed rows (rows past cu[-1] hold anything)."""
        x = self.embed[tokens.clamp(min=0).long()]
        heads = (self.Hq, self.Hkv, self.Hkv)
        for i, w in enumerate(self.layers):
            q, k, v = (self.norm(x) @ w["qkv"].t()).view(-1, sum(heads), self.D).split(heads, 1)
            q = dspark.dspark_append_kv(q, k, v, self.cos, self.sin, cu, ctx, table, self.k[i],
                                        self.v[i], k_scale=self.scale, v_scale=self.scale)
            o = torch.zeros_like(q)
            dspark.dspark_verify_attention(q, self.k[i], self.v[i], cu, ctx, table, max_rows,
                                           k_scale=self.scale, v_scale=self.scale, out=o)
            x = x + o.flatten(1) @ w["o"].t()
            x = x + torch.relu(self.norm(x) @ w["up"].t()) @ w["down"].t()
        return self.norm(x) @ self.head.t()


class Loop:
    """A batch of requests: `step()` verifies one block of drafts per request."""

    def __init__(self, target, prompts, gamma=4, temperature=0.7, top_k=40, top_p=0.95, seed=1):
        t, dev, B = target, target.device, len(prompts)
        self.target, self.gamma, self.B = t, gamma, B
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        width = t.k.shape[1] // B
        order = torch.randperm(t.k.shape[1], generator=self.gen, device=dev).to(I32)
        self.table = order[:B * width].view(B, width).contiguous()
        self.ctx = torch.zeros(B, dtype=I32, device=dev)
        f = lambda v: torch.full((B,), v, dtype=torch.float32, device=dev)  # noqa: E731
        self.sampling = dict(temperature=f(temperature), top_p=f(top_p), min_p=f(0.0),
                             top_k=torch.full((B,), top_k, dtype=I32, device=dev))
        # the drafter: the next token by the embedding alone, sure of itself by a random head
        self.next = (t.norm(t.embed) @ t.head.t()).argmax(1).to(I32)
        self.w = (torch.randn(t.embed.shape[1], generator=self.gen, device=dev) * 0.2).to(BF16)
        self.temps = torch.ones(gamma, device=dev)
        self.cutoff = f(0.2)
        self.uniforms = torch.rand(B * (gamma + 1), generator=self.gen, device=dev)
        self.tokens = torch.zeros((B, gamma + 1), dtype=I32, device=dev)
        self.root = self._prompts(prompts)

    def _prompts(self, prompts):
        """The prompts as packed chunks; returns each request's first drawn token."""
        dev = self.target.device
        lens = [len(p) for p in prompts]
        cu = torch.tensor([0] + lens, device=dev).cumsum(0).to(I32)
        tokens = torch.tensor([t for p in prompts for t in p], dtype=I32, device=dev)
        logits = self.target.forward(tokens, cu, self.ctx, self.table, max(lens))
        last = logits[(cu[1:] - 1).long()]
        # one row per request in a block of gamma + 1, nothing drafted
        block = last.repeat_interleave(self.gamma + 1, 0)
        ones = torch.arange(self.B + 1, dtype=I32, device=dev)
        src = torch.full((self.B * (self.gamma + 1),), -1, dtype=I32, device=dev)
        src[:self.B] = torch.arange(self.B, device=dev).to(I32) * (self.gamma + 1)
        _, _, bonus = dspark.dspark_sample_accept(block, src, ones, self.tokens, self.uniforms,
                                                  **self.sampling)
        self.ctx += torch.tensor(lens, dtype=I32, device=dev)
        return bonus.clone()

    def step(self):
        """Drafts, verifies and commits; returns (tokens, lengths, accepted, bonus, logits, cu)."""
        self.tokens[:, 0] = self.root
        for j in range(self.gamma):
            self.tokens[:, j + 1] = self.next[self.tokens[:, j].long()]
        hidden = self.target.embed[self.tokens[:, 1:].long()]
        _, survival = dspark.dspark_confidence(hidden, self.w, 1.5, self.temps)
        lengths = dspark.dspark_schedule(survival, "threshold", cutoff=self.cutoff)
        cu, packed, _, _ = dspark.dspark_compact(lengths, self.tokens)
        logits = self.target.forward(packed, cu, self.ctx, self.table, self.gamma + 1)
        drawn, accepted, bonus = dspark.dspark_sample_accept(
            logits, None, cu, self.tokens, self.uniforms, **self.sampling)
        self.ctx += accepted + 1  # the root and the accepted drafts are in the cache
        self.root.copy_(bonus)
        return self.tokens, lengths, accepted, bonus, logits, cu

    def new_numbers(self):
        self.uniforms.uniform_(generator=self.gen)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--graph", action="store_true", help="capture a step and replay it")
    a = ap.parse_args()
    prompts, gamma, page = [[5, 17, 300], list(range(40, 90)), [7] * 20, [999]], 4, 16
    # rows past the angles' tables or the requests' pages would be left out
    longest = max(len(p) for p in prompts) + a.steps * (gamma + 1)
    target = Target(cache=BF16 if a.cache == "bf16" else torch.float8_e4m3fn, page=page,
                    pages=max(512, len(prompts) * -(-longest // page)), longest=max(1024, longest))
    loop = Loop(target, prompts, gamma)
    out = [[t] for t in loop.root.tolist()]
    run = loop.step
    if a.graph:
        keep = [loop.ctx.clone(), loop.root.clone()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # a step outside the graph allocates what steps share
            loop.step()
        torch.cuda.current_stream().wait_stream(side)
        loop.ctx.copy_(keep[0])
        loop.root.copy_(keep[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = loop.step()

        def run():
            graph.replay()
            return held
    drafted = taken = 0
    for _ in range(a.steps):
        loop.new_numbers()
        tokens, lengths, accepted, bonus, _, _ = run()
        rows = zip(tokens.tolist(), accepted.tolist(), bonus.tolist())
        for b, (block, n, last) in enumerate(rows):
            out[b] += block[1:1 + n] + [last]
        drafted += int(lengths.sum())
        taken += int(accepted.sum())
    for b, seq in enumerate(out):
        print(f"request {b}: {len(seq)} tokens, the first {seq[:10]}")
    print(f"{a.steps} steps, {taken} of {drafted} drafts accepted")


if __name__ == "__main__":
    main()
