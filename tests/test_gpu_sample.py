"""Drawing the target's tokens and accepting the drafts against the 64-bit
definition, token for token (needs an MI355X): every filter, ties, masks,
infinities and NaN, odd vocabularies, dense and packed logits, refilled
buffers, graph replays."""
import numpy as np
import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
import forward_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def make(B, g, V, seed, std=1.4, ties=False, dense=True, filters="mixed"):
    rng = np.random.default_rng(seed)
    cap = B * (g + 1)
    x = rng.normal(0, std, (cap, V))
    if ties:
        x = np.round(x * 2) / 2
    logits = torch.from_numpy(x).bfloat16()
    tokens = rng.integers(0, V, (B, g + 1))
    rows = rng.integers(1, g + 2, B)
    cu = np.concatenate([[0], np.cumsum(rows)])
    psrc = np.full(cap, -1)
    r = 0
    for b in range(B):
        for j in range(rows[b]):
            psrc[r] = b * (g + 1) + j
            r += 1
    at = psrc[:r] if dense else np.arange(r)
    pick = dict(mixed=((0.0, 0.6, 1.0, 1.7), (0, 1, 20, 5 * V), (1.0, 0.95, 0.5, 0.01),
                       (0.0, 0.05, 0.5)),
                none=((1.0,), (0,), (1.0,), (0.0,)), all=((0.7,), (40,), (0.9,), (0.02,)))[filters]
    c = dict(logits=logits, tokens=tokens, cu=cu, psrc=psrc if dense else None,
             uniforms=rng.random(cap).astype(np.float32),
             temperature=rng.choice(pick[0], B).astype(np.float32), top_k=rng.choice(pick[1], B),
             top_p=rng.choice(pick[2], B).astype(np.float32),
             min_p=rng.choice(pick[3], B).astype(np.float32))
    # drafts that the drawn tokens often agree with
    drawn = ref.sample_accept(logits.double().numpy(), c["psrc"], cu, tokens, c["uniforms"],
                              c["temperature"], c["top_k"], c["top_p"], c["min_p"])[0]
    for b in range(B):
        for j in range(rows[b] - 1):
            if rng.random() < 0.7:
                tokens[b, j + 1] = drawn[cu[b] + j]
    assert at.size == r
    return c


def dev(c, key, dtype):
    return None if c[key] is None else torch.from_numpy(np.ascontiguousarray(c[key])).to(dtype).to(DEV)


def call(c, logits=None, **kw):
    i32, f32 = torch.int32, torch.float32
    return dspark.dspark_sample_accept(
        c["logits"].to(DEV) if logits is None else logits, dev(c, "psrc", i32), dev(c, "cu", i32),
        dev(c, "tokens", i32), dev(c, "uniforms", f32), temperature=dev(c, "temperature", f32),
        top_k=dev(c, "top_k", i32), top_p=dev(c, "top_p", f32), min_p=dev(c, "min_p", f32), **kw)


def check(c, logits=None):
    want = ref.sample_accept(c["logits"].double().numpy(), c["psrc"], c["cu"], c["tokens"],
                             c["uniforms"], c["temperature"], c["top_k"], c["top_p"], c["min_p"])
    got = call(c, logits)
    torch.cuda.synchronize()
    for name, g, w in zip(("packed_sample", "accepted", "bonus"), got, want):
        g = g.cpu().numpy()
        assert np.array_equal(g, w), (name, np.nonzero(g != w)[0][:5], g[g != w][:5], w[g != w][:5])


@pytest.mark.parametrize("V", [1, 2, 7, 64, 1000, 1001, 8192, 32003, 151936])
@pytest.mark.parametrize("dense", [True, False])
def test_vocabularies(V, dense):
    check(make(5, 3, V, seed=V, dense=dense))


@pytest.mark.parametrize("filters", ["none", "all", "mixed"])
@pytest.mark.parametrize("ties", [False, True])
def test_filters_and_ties(filters, ties):
    for seed in range(4):
        check(make(12, 5, 4096, seed=seed, ties=ties, filters=filters))


@pytest.mark.parametrize("std", [1e-3, 0.1, 10.0, 1000.0, 1e30])
def test_spreads(std):
    check(make(16, 4, 5000, seed=11, std=std))
    check(make(16, 4, 5000, seed=12, std=std, filters="none"))


def test_drafts_are_accepted():
    c = make(40, 6, 512, seed=3)
    acc = call(c)[1].cpu().numpy()
    assert acc.max() >= 3
    check(c)


@pytest.mark.parametrize("mask", [float("-inf"), -3.3895313892515355e38, -65504.0, -1e9,
                                  float("nan")])
def test_masked_vocabularies(mask):
    """All but a few entries masked, as constrained decoding leaves them."""
    c = make(24, 4, 70001, seed=21)
    keep = torch.rand(c["logits"].shape, generator=torch.Generator().manual_seed(1)) < 2e-4
    keep[:, 70000] = True
    c["logits"] = torch.where(keep, c["logits"], torch.full_like(c["logits"], mask))
    check(c)


@pytest.mark.parametrize("value", [0.0, 1.5, -3.3895313892515355e38, -2.0 ** -30])
@pytest.mark.parametrize("V", [1000, 140001])
def test_rows_of_one_value(value, V):
    c = make(6, 2, V, seed=22, filters="mixed")
    c["logits"].fill_(value)
    check(c)


def test_rows_with_nothing_and_with_infinities():
    c = make(20, 3, 3000, seed=23)
    c["logits"][::4] = float("-inf")
    c["logits"][1::4] = float("nan")
    c["logits"][2::8, 100:105] = float("inf")
    c["logits"][3::8, ::2] = float("nan")
    c["logits"][6::8, 2900] = float("inf")
    check(c)


def test_signed_zeros_are_equal():
    c = make(12, 3, 2048, seed=24, filters="none")
    x = torch.where(torch.rand(c["logits"].shape, generator=torch.Generator().manual_seed(2)) < 0.5,
                    torch.tensor(-0.0), torch.tensor(0.0))
    c["logits"] = x.bfloat16()
    check(c)


def test_small_magnitudes():
    """Values across the whole exponent range in one row."""
    rng = np.random.default_rng(5)
    c = make(16, 3, 6000, seed=25, filters="mixed")
    x = rng.normal(0, 1, (64, 6000)) * 10.0 ** rng.uniform(-38, 1, (64, 6000))
    c["logits"] = torch.from_numpy(x).bfloat16()
    check(c)
    x = np.abs(rng.normal(0, 1, (64, 6000))) * 10.0 ** rng.uniform(-38, 38, (64, 6000))
    c["logits"] = torch.from_numpy(x).bfloat16()
    check(c)


@pytest.mark.parametrize("T", [1e-30, 1e-3, 50.0, 1e6, 1e38])
def test_extreme_temperatures(T):
    c = make(10, 3, 4000, seed=26, std=4.0)
    c["temperature"][:] = T
    c["logits"][:, ::3] = -1e9
    check(c)


def test_ends_of_the_uniform_range():
    c = make(16, 3, 4000, seed=27, filters="mixed")
    c["uniforms"][::2] = 0.0
    c["uniforms"][1::2] = 1.0 - 2.0 ** -24
    check(c)


def test_no_filters_given():
    c = make(6, 3, 2000, seed=28, filters="none")
    c["temperature"] = c["top_k"] = c["top_p"] = c["min_p"] = None
    check(c)


def test_source_rows_outside_the_block():
    c = make(8, 3, 1000, seed=29)
    total = int(c["cu"][-1])
    c["psrc"][1:total:3] = -1
    c["psrc"][2:total:5] = 32
    check(c)


def test_requests_without_rows():
    c = make(6, 3, 1000, seed=30)
    c["cu"] = np.array([0, 0, 2, 2, 3, 3, 3])
    check(c)


def test_misaligned_logits():
    c = make(4, 3, 1000, seed=31)
    flat = torch.zeros(c["logits"].numel() + 1, dtype=torch.bfloat16, device=DEV)
    flat[1:] = c["logits"].reshape(-1).to(DEV)
    check(c, flat[1:].view(c["logits"].shape))


@pytest.mark.parametrize("V", [1024, 50001])
def test_greedy_is_dspark_accept(V):
    c = make(30, 5, V, seed=32, ties=True)
    c["temperature"][:] = 0.0
    got = call(c)
    i32 = torch.int32
    want = dspark.dspark_accept(c["logits"].to(DEV), dev(c, "psrc", i32), dev(c, "cu", i32),
                                dev(c, "tokens", i32))
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_more_requests_than_one_launch_of_the_step():
    c = make(4200, 1, 50, seed=33)
    check(c)


def test_shares_the_workspace_with_accept():
    c = make(30, 5, 2000, seed=34)
    ws = dspark.workspace(30, 5, 2000, DEV)
    i32 = torch.int32
    first = [t.clone() for t in call(c, ws=ws)]
    dspark.dspark_accept(c["logits"].to(DEV), dev(c, "psrc", i32), dev(c, "cu", i32),
                         dev(c, "tokens", i32), ws=ws)
    again = call(c, ws=ws)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_graph_replays_match_eager():
    cases = [make(12, 4, 3001, seed=40 + i) for i in range(3)]
    i32, f32 = torch.int32, torch.float32
    kinds = dict(psrc=i32, cu=i32, tokens=i32, uniforms=f32, temperature=f32, top_k=i32, top_p=f32,
                 min_p=f32)
    buf = {k: dev(cases[0], k, d).clone() for k, d in kinds.items()}
    logits = cases[0]["logits"].to(DEV)
    out = dict(packed_sample=torch.full((60,), -1, dtype=i32, device=DEV),
               accepted=torch.zeros(12, dtype=i32, device=DEV),
               bonus=torch.zeros(12, dtype=i32, device=DEV))

    def body():
        dspark.dspark_sample_accept(logits, buf["psrc"], buf["cu"], buf["tokens"], buf["uniforms"],
                                    buf["temperature"], buf["top_k"], buf["top_p"], buf["min_p"],
                                    out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for c in cases * 2:
        for k, d in kinds.items():
            buf[k].copy_(dev(c, k, d))
        logits.copy_(c["logits"])
        out["packed_sample"].fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        eager = call(c)
        for g, w in zip((out["packed_sample"], out["accepted"], out["bonus"]), eager):
            assert torch.equal(g, w)


def fill(c, value, where):
    c["logits"] = torch.where(where, torch.tensor(value).bfloat16(), c["logits"])


@pytest.mark.parametrize("V", [140001, 262147])
@pytest.mark.parametrize("greedy", [False, True])
def test_more_equals_than_16_bits_count(V, greedy):
    """One value 65536 times and more in either half of a row, or in one of them."""
    for lo, hi in ((0, V), (0, 65536), (V - 65536, V), (3, 65535 + 3), (V // 2, V)):
        c = make(2, 1, V, seed=50, filters="none")
        if greedy:
            c["temperature"][:] = 0.0
        at = torch.arange(V)
        fill(c, 20.0, ((at >= lo) & (at < hi))[None].expand(c["logits"].shape))
        check(c)


@pytest.mark.parametrize("V", [4099, 150001])
def test_more_equals_than_are_listed(V):
    """A drawn value with over a thousand equals, whose order decides."""
    c = make(20, 2, V, seed=51, filters="none")
    c["logits"] = (torch.round(c["logits"].float() / 2) * 2).bfloat16()
    check(c)


@pytest.mark.parametrize("value", [65280.0, 65536.0, -65536.0, 2.0 ** -32, -2.0 ** -33, 2.0 ** -40,
                                   float("inf"), float("nan")])
@pytest.mark.parametrize("T", [0.0, 1.0, 3000.0])
def test_values_at_the_ends_of_the_counted_range(value, T):
    c = make(9, 2, 3001, seed=52, filters="mixed")
    c["temperature"][:] = T
    at = torch.rand(c["logits"].shape, generator=torch.Generator().manual_seed(3)) < 0.01
    at[::3] = False
    fill(c, value, at)
    check(c)
    c["logits"] = -c["logits"]
    check(c)


@pytest.mark.parametrize("V", [1, 3, 9, 15, 23, 1003])
@pytest.mark.parametrize("T", [0.0, 1.0])
def test_the_last_entries_of_rows_at_every_alignment(V, T):
    c = make(16, 1, V, seed=53, filters="none")
    c["temperature"][:] = T
    for i in range(c["logits"].shape[0]):
        c["logits"][i, V - 1 - i % min(V, 9)] = 30.0
    check(c)


def test_a_masked_vocabulary_over_16_bits():
    for mask in (float("-inf"), -3.3895313892515355e38, -1e9):
        c = make(3, 2, 200003, seed=54)
        keep = torch.rand(c["logits"].shape, generator=torch.Generator().manual_seed(4)) < 1e-4
        keep[:, 5] = True
        fill(c, mask, ~keep)
        check(c)


def test_lengths_out_of_order_leave_the_workspace_as_it_was():
    """cu_seqlens that go down give every row one owner; the next call is right."""
    c = make(40, 4, 700, seed=55)
    good = c["cu"]
    ws = torch.zeros(dspark.dspark_workspace_bytes(40, 4, 700), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(56)
    for _ in range(4):
        c["cu"] = rng.integers(-3, 205, 41)
        call(c, ws=ws)
        torch.cuda.synchronize()
    c["cu"] = good
    want = ref.sample_accept(c["logits"].double().numpy(), c["psrc"], c["cu"], c["tokens"],
                             c["uniforms"], c["temperature"], c["top_k"], c["top_p"], c["min_p"])
    for g, w in zip(call(c, ws=ws), want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert int(ws.sum()) == 0
