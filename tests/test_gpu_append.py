"""Appending rotated keys and values to the paged cache against its 64-bit
definition (needs an MI355X): head layouts, types, page sizes, strided inputs
and pools, rows without a page, rows past the packed total."""
import random

import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
import forward_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def make(B, rows, Hq, Hkv, D, page, cache="bf16", rot=None, seed=0, ctx_hi=200, spare=3,
         layout="page_head", holes=False, offset=0):
    """CPU tensors of one call. layout: the pool's axes; `offset` elements of
    misalignment of the fused projection and the pools."""
    rng, gen = random.Random(seed), torch.Generator().manual_seed(seed)
    rot = D if rot is None else rot
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    ctx = [rng.randint(0, ctx_hi) for _ in range(B)]
    need = [-(-(c + n) // page) for c, n in zip(ctx, rows)]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32)
    used = 0
    for b in range(B):
        for i in range(need[b]):
            table[b, i] = perm[used]
            used += 1
    if holes:
        for b in range(0, B, 2):
            table[b, need[b] - 1] = [-1, pages, pages + 7, -5][b // 2 % 4]
    cap = cu[-1] + 2
    flat = torch.randn(cap * (Hq + 2 * Hkv) * D + offset, generator=gen).bfloat16()
    longest = max(c + n for c, n in zip(ctx, rows))
    half = rot // 2
    ang = torch.arange(longest, dtype=torch.float64)[:, None] * 1000.0 ** (
        -torch.arange(half, dtype=torch.float64) / max(half, 1))
    dtype = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    order = dict(page_head=(pages, Hkv, page, D), page_slot=(pages, page, Hkv, D))[layout]
    n = pages * Hkv * page * D

    def pool():
        x = torch.randn(n + offset, generator=gen) * (20 if cache == "e4m3" else 1)
        return x.to(dtype)
    return dict(flat=flat, cap=cap, cos=ang.cos().float(), sin=ang.sin().float(), cu=cu, ctx=ctx,
                table=table, kf=pool(), vf=pool(), order=order, layout=layout, offset=offset,
                Hq=Hq, Hkv=Hkv, D=D)


def views(c, dev):
    off = c["offset"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    flat = c["flat"].to(dev)
    q, k, v = flat[off:].view(c["cap"], Hq + 2 * Hkv, D).split((Hq, Hkv, Hkv), 1)

    def pool(x):
        x = (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x).to(dev)
        if c["kf"].dtype == torch.float8_e4m3fn:
            x = x.view(torch.float8_e4m3fn)
        x = x[off:].view(c["order"])
        return x if c["layout"] == "page_head" else x.transpose(1, 2)
    return q, k, v, pool(c["kf"]), pool(c["vf"])


def check(c, interleaved=False, k_scale=1.0, v_scale=1.0, poison=False):
    q, k, v, kc, vc = views(c, "cpu")
    out = torch.randn(q.shape).bfloat16()
    O, K, V, ot, kt, vt = ref.append(q, k, v, c["cos"], c["sin"], c["cu"], c["ctx"], c["table"],
                                     kc, vc, interleaved, k_scale, v_scale, out)
    gq, gk, gv, gkc, gvc = views(c, DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    got = dspark.dspark_append_kv(gq, gk, gv, c["cos"].to(DEV), c["sin"].to(DEV), i32(c["cu"]),
                                  i32(c["ctx"]), c["table"].to(DEV), gkc, gvc,
                                  interleaved=interleaved, k_scale=k_scale, v_scale=v_scale,
                                  out=out.to(DEV))
    torch.cuda.synchronize()
    for name, g, want, tol in (("q", got, O, ot), ("k", gkc, K, kt), ("v", gvc, V, vt)):
        g = g.cpu().double()
        assert torch.equal(torch.isnan(g), torch.isnan(want)), name
        bad = (g - want).abs() > tol
        assert not bool(bad.any()), (name, int(bad.sum()), float((g - want).abs().max()))


@pytest.mark.parametrize("Hq,Hkv,D,page,rot,interleaved", [
    (8, 2, 128, 16, 128, False), (8, 2, 128, 16, 64, True), (5, 1, 64, 32, 64, False),
    (6, 3, 64, 64, 32, True), (4, 4, 128, 128, 128, True), (3, 1, 80, 16, 80, False),
    (2, 2, 96, 24, 64, False), (4, 2, 256, 16, 128, False), (4, 2, 72, 16, 36, False),
    (4, 2, 66, 7, 66, True), (2, 1, 128, 1, 0, False), (1, 1, 2, 3, 2, False)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_layouts(Hq, Hkv, D, page, rot, interleaved, cache):
    c = make(5, [1, 7, 0, 17, 3], Hq, Hkv, D, page, cache, rot, seed=Hq + D)
    check(c, interleaved, 0.03125, 0.0234375)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout,offset", [("page_slot", 0), ("page_head", 1), ("page_slot", 8)])
def test_strides_and_alignment(cache, layout, offset):
    check(make(3, [2, 1, 5], 8, 2, 64, 16, cache, layout=layout, offset=offset, seed=3), False,
          0.5, 0.25)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_rows_without_a_page(cache):
    check(make(8, [3] * 8, 4, 2, 64, 16, cache, holes=True, seed=4), True, 0.1, 0.3)


def test_many_requests():
    check(make(300, [1 + i % 3 for i in range(300)], 2, 1, 64, 16, seed=5, ctx_hi=40))


def test_prompt_rows():
    check(make(2, [130, 77], 4, 1, 128, 32, "e4m3", seed=6, ctx_hi=0), False, 0.02, 0.02)


def test_values_past_the_range_and_nan():
    c = make(2, [4, 4], 2, 1, 64, 16, "e4m3", seed=7)
    c["flat"][::5] = 3000.0
    c["flat"][1::7] = -9000.0
    c["flat"][3::41] = float("nan")
    check(c, False, 0.5, 0.5)


def test_positions_past_the_tables():
    c = make(2, [6, 6], 2, 1, 64, 16, seed=8)
    keep = max(c["ctx"]) + 2
    c["cos"], c["sin"] = c["cos"][:keep].contiguous(), c["sin"][:keep].contiguous()
    check(c)


def test_rotation_in_place():
    c = make(2, [6, 3], 4, 2, 128, 16, seed=9)
    q, k, v, kc, vc = views(c, DEV)
    q = q.contiguous()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    args = (c["cos"].to(DEV), c["sin"].to(DEV), i32(c["cu"]), i32(c["ctx"]), c["table"].to(DEV))
    apart = dspark.dspark_append_kv(q, k, v, *args, kc, vc, out=q.clone())
    same = dspark.dspark_append_kv(q, k, v, *args, kc, vc, out=q)
    assert same is q
    assert torch.equal(apart, q)


def test_on_another_stream():
    c = make(4, [5, 1, 9, 2], 8, 2, 128, 16, seed=10)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        check(c)
    torch.cuda.synchronize()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_pool_past_32_bits(cache):
    """The last pages of pools of over 2^32 bytes."""
    Hq, Hkv, D, page = 4, 2, 128, 16
    item = 1 if cache == "e4m3" else 2
    dtype = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    pages = 5 * 2 ** 30 // (Hkv * page * D * item)
    gen = torch.Generator().manual_seed(7)
    x = torch.randn((3, Hq + 2 * Hkv, D), generator=gen).bfloat16()
    q, k, v = x.split((Hq, Hkv, Hkv), 1)
    angle = torch.rand((40, D // 2), generator=gen) * 6
    cos, sin = angle.cos(), angle.sin()
    cu, ctx = [0, 3], [30]
    small = torch.zeros((4, Hkv, page, D)).to(dtype)
    table = torch.tensor([[0, 2, 3]], dtype=torch.int32)
    out = torch.zeros((3, Hq, D)).bfloat16()
    scale = dict(k_scale=0.01, v_scale=0.02) if item == 1 else {}
    O, K, V, ot, kt, vt = ref.append(q, k, v, cos, sin, cu, ctx, table, small, small, out=out,
                                     **scale)
    pools = [torch.empty((pages, Hkv, page, D), dtype=torch.uint8 if item == 1 else dtype,
                         device=DEV) for _ in range(2)]
    for p in pools:
        p[pages - 4:] = 0
    kc, vc = (p.view(dtype) for p in pools)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    got = dspark.dspark_append_kv(*(t.to(DEV) for t in (x[:, :Hq], x[:, Hq:Hq + Hkv],
                                                        x[:, Hq + Hkv:])),
                                  cos.to(DEV), sin.to(DEV), i32(cu), i32(ctx),
                                  (table + pages - 4).to(DEV), kc, vc, **scale)
    torch.cuda.synchronize()
    ends = [p[pages - 4:].cpu().view(dtype).double() for p in pools]
    del pools, kc, vc
    assert bool(((got.cpu().double() - O).abs() <= ot).all())
    assert bool(((ends[0] - K).abs() <= kt).all()) and bool(((ends[1] - V).abs() <= vt).all())
    torch.cuda.empty_cache()
