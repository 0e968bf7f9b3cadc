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
    monkeypatch.setattr(dspark, "_capture_id", lambda device: 0)
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



@pytest.mark.parametrize("entry,sizes", KEPT)
def test_a_workspace_made_in_a_capture_is_not_for_other_calls(on_cpu, monkeypatch, entry, sizes):
    """Its zero-fill only runs with the graph, so a call outside must not take it."""
    dev = "cpu:%d" % (8 + KEPT.index((entry, sizes)))
    capture = [0]
    monkeypatch.setattr(dspark, "_capture_id", lambda device: capture[0])
    small, middle, large = sizes
    at = lambda s: entry(*s, dev).data_ptr()  # noqa: E731
    capture[0] = 5
    inside = entry(*middle, dev)
    assert at(middle) == at(small) == inside.data_ptr()   # one for all calls of a capture
    capture[0] = 0
    eager = entry(*small, dev)
    assert eager.data_ptr() != inside.data_ptr()
    capture[0] = 6                                        # another graph, replayed before the first
    assert at(small) == eager.data_ptr()                  # one that calls outside have zeroed serves
    assert at(large) not in (eager.data_ptr(), inside.data_ptr())
    capture[0] = 0
    assert at(large) != inside.data_ptr() and at(small) == at(large)


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
def test_a_capture_without_a_call_before_it(monkeypatch):
    """Eager calls before the first replay, between replays and after the graph is gone."""
    args, want = sample_inputs(6, 4, 300, 1)
    zeros = torch.zeros(dspark.dspark_workspace_bytes(6, 4, 300), dtype=torch.uint8, device="cuda:0")
    assert same(dspark.dspark_sample_accept(*args, ws=zeros), want)  # loads the kernels
    monkeypatch.setattr(dspark, "_WS", {})
    out = {k: torch.zeros(n, dtype=torch.int32, device="cuda:0")
           for k, n in (("packed_sample", 30), ("accepted", 6), ("bonus", 6))}
    graph, _ = captured(lambda: [dspark.dspark_sample_accept(*args, out=out) for _ in range(3)])
    assert same(dspark.dspark_sample_accept(*args), want)
    for _ in range(3):
        for x in out.values():
            x.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out.values(), want)
        assert same(dspark.dspark_sample_accept(*args), want)
    del graph
    torch.cuda.synchronize()
    assert same(dspark.dspark_sample_accept(*args), want)


@pytest.mark.gpu
def test_a_captured_attention_without_a_call_before_it(monkeypatch):
    """A context split between workgroups, whose partial results and arrivals need zeros."""
    gen = torch.Generator(device="cuda:0").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda:0").bfloat16()  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda:0")  # noqa: E731
    q, k, v = r(1, 8, 128), r(70, 2, 64, 128), r(70, 2, 64, 128)
    args = (q, k, v, i32(0, 1), i32(4100), torch.arange(70, dtype=torch.int32, device="cuda:0")[None], 1)
    ws = torch.zeros(dspark.dspark_attention_workspace_bytes(1, 1, 8, 2, 128), dtype=torch.uint8,
                     device="cuda:0")
    want = dspark.dspark_verify_attention(*args, ws=ws)
    monkeypatch.setattr(dspark, "_ATTN_WS", {})
    out = torch.zeros_like(want)
    graph, _ = captured(lambda: [dspark.dspark_verify_attention(*args, out=out) for _ in range(3)])
    assert torch.equal(dspark.dspark_verify_attention(*args), want)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(dspark.dspark_verify_attention(*args), want)


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
