"""Lifetime of the workspaces that the binding keeps for calls without one of
their own: on the CPU by the tensors themselves, on the GPU by captured graphs."""
import os
import weakref

import numpy as np
import pytest
import torch

import __graft_entry__
import confidence_scheduled_ragged_amd as dspark

# (entry, arguments of rising need)
KEPT = [(dspark.workspace, [(1, 4, 100), (64, 4, 100), (256, 4, 100)]),
        (dspark.attention_workspace, [(1, 1, 8, 8, 64), (1, 16, 32, 8, 64), (1, 32, 32, 8, 128)])]


@pytest.fixture
def on_cpu(monkeypatch):
    """The binding's workspaces made on the CPU, zero-filled by torch."""
    if not os.path.exists(dspark.LIB_PATH):
        __graft_entry__.build()
    monkeypatch.setattr(dspark, "dspark_workspace_init", lambda ws: ws.zero_())
    return "cpu:7"  # a device that no other test uses


@pytest.mark.parametrize("entry,sizes", KEPT)
def test_an_outgrown_workspace_stays_allocated(on_cpu, entry, sizes):
    made = []
    for s in sizes:
        ws = entry(*s, on_cpu)
        made.append((weakref.ref(ws), ws.data_ptr(), ws.numel()))
        del ws
    assert [n for _, _, n in made] == sorted({n for _, _, n in made})
    assert all(w() is not None for w, _, _ in made)
    # a smaller call takes the newest
    assert entry(*sizes[0], on_cpu).data_ptr() == made[-1][1]


def sample_inputs(B, g, V, seed, dev="cuda:0"):
    """A batch of whole windows whose drafts sometimes agree; the oracle's answer beside it."""
    import forward_ref as ref
    rng = np.random.default_rng(seed)
    logits = torch.from_numpy(rng.normal(0, 2, (B * (g + 1), V))).bfloat16()
    tokens = rng.integers(0, V, (B, g + 1))
    cu = np.arange(B + 1) * (g + 1)
    u = rng.random(B * (g + 1)).astype(np.float32)
    want = ref.sample_accept(logits.double().numpy(), None, cu, tokens, u)
    i32 = lambda x: torch.from_numpy(x).to(torch.int32).to(dev)  # noqa: E731
    return (logits.to(dev), None, i32(cu), i32(tokens), torch.from_numpy(u).to(dev)), want


def same(got, want):
    return all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want))


def captured(body):
    """body() in a graph; kernels are loaded before by a call of the caller's."""
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = body()
    return graph, held


@pytest.mark.gpu
def test_a_graph_outlives_the_growth_of_its_workspace(monkeypatch):
    """Graphs captured for batches that grow: each keeps the workspace it was
    captured with, and no later tensor lies in it."""
    monkeypatch.setattr(dspark, "_WS", {})
    graphs = []
    for B in (1, 64, 256):
        args, want = sample_inputs(B, 4, 300, B)
        assert same(dspark.dspark_sample_accept(*args), want)
        out = dict(zip(("packed_sample", "accepted", "bonus"),
                       (torch.zeros(n, dtype=torch.int32, device="cuda:0")
                        for n in (B * 5, B, B))))
        graph, _ = captured(lambda: dspark.dspark_sample_accept(*args, out=out))
        graphs.append((graph, args, out, want))
    need = dspark.dspark_workspace_bytes(1, 4, 300)
    later = [torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda:0") for _ in range(16)]
    for _ in range(3):
        for graph, args, out, want in graphs:
            for x in out.values():
                x.fill_(-7)
            graph.replay()
            torch.cuda.synchronize()
            assert same(out.values(), want)
            assert same(dspark.dspark_sample_accept(*args), want)
    assert all(bool((x == 0x5A).all()) for x in later)
