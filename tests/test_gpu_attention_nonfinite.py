"""NaN and infinities that a row does see reach its result however its positions
are divided between workgroups and joined again (needs an MI355X)."""
import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark  # noqa: F401
import forward_ref as ref
from test_gpu_attention import DEV, SCALES, call, make, pools

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# head size, cache, positions of a tile (of a step of the row kernel over 128)
HEADS = [(64, "bf16", 128), (128, "bf16", 64), (96, "bf16", 64), (64, "e4m3", 256),
         (128, "e4m3", 128), (136, "bf16", 64), (192, "e4m3", 64)]


def run(c, cache, **kw):
    out = torch.zeros((c["cap"], c["Hq"], c["D"]), dtype=torch.bfloat16, device=DEV)
    got = call(c, *pools(c, DEV), out, **SCALES[cache], **kw)
    torch.cuda.synchronize()
    return got.cpu().float()


def poison(c, pool, b, positions, value, elements=slice(None)):
    """Sets elements of every head at positions of request b."""
    raw = torch.tensor(value).to(c[pool].dtype).view(
        torch.uint8 if c[pool].dtype == torch.float8_e4m3fn else torch.int16)
    page = c[pool].shape[2]
    flat = c[pool].view(raw.dtype)
    for t in positions:
        flat[int(c["table"][b, t // page]), :, t % page, elements] = raw


@pytest.mark.parametrize("D,cache,keys", HEADS)
@pytest.mark.parametrize("rows,ctx", [([1], [4000]), ([17], [4000]), ([150, 2], [2000, 70]),
                                      ([1], [0]), ([3, 1], [5, 300])])
def test_a_query_that_is_nan(D, cache, keys, rows, ctx):
    """All scores of one query row are NaN: so is its result, and only its result."""
    c = make(rows, ctx, 8, 2, D, 16, cache, seed=30)
    clean = run(c, cache)
    hits = [(0, 3), (c["cu"][1] - 1, 0)]
    for r, h in hits:
        c["q"][r, h, 5] = NAN
    got = run(c, cache)
    for r, h in hits:
        assert bool(got[r, h].isnan().all())
        got[r, h] = clean[r, h]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("D,cache,keys", HEADS)
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 2)])
def test_keys_that_are_nan(D, cache, keys, Hq, Hkv):
    """One key alone in the last tile, the first tile whole, a tile within, all of them."""
    ctx = 65 * keys
    for hit in (range(ctx, ctx + 1), range(keys), range(30 * keys, 31 * keys), range(ctx + 1)):
        c = make([1], [ctx], Hq, Hkv, D, 16, cache, seed=31)
        poison(c, "kc", 0, hit, NAN, slice(4, 5))
        assert bool(run(c, cache)[0].isnan().all()), hit


@pytest.mark.parametrize("D,cache,keys", HEADS)
@pytest.mark.parametrize("value", [NAN, INF])
def test_values_whose_weight_is_nothing_beside_the_others(D, cache, keys, value):
    """Later keys score so far above that the earlier weights are 0 in 32 bits: zero
    times an infinity is NaN, in the elements that hold it."""
    ctx = 40 * keys
    c = make([1], [ctx], 8, 8, D, 16, cache, seed=32)
    for t in range(39 * keys, ctx + 1):
        c["kc"][int(c["table"][0, t // 16]), :, t % 16] = (
            c["q"][0].float() * (20.0 if cache == "bf16" else 400.0)).clamp(-448, 448).to(c["kc"].dtype)
    clean = run(c, cache)
    assert bool(clean[0].isfinite().all())
    poison(c, "vc", 0, [3], value, slice(2, None, 7))
    got = run(c, cache)[0]
    assert not bool(got[:, 2::7].isfinite().any())
    keep = [d for d in range(D) if d % 7 != 2]
    assert torch.equal(got[:, keep], clean[0][:, keep])


@pytest.mark.parametrize("D,cache,keys", HEADS)
def test_values_that_are_nan_in_a_tile_of_their_own(D, cache, keys):
    ctx = 65 * keys
    for hit in ([ctx], range(keys), range(64 * keys, 65 * keys)):
        c = make([1], [ctx], 8, 8, D, 16, cache, seed=33)
        poison(c, "vc", 0, hit, NAN, slice(1, None, 3))
        got = run(c, cache)[0]
        assert bool(got[:, 1::3].isnan().all())
        assert bool(got[:, 0::3].isfinite().all())


@pytest.mark.parametrize("D,cache,keys", HEADS)
@pytest.mark.parametrize("rows", [2, 17])
def test_every_row_of_a_tile_seen_in_part(D, cache, keys, rows):
    """A value that is NaN at one position of the last tile, wherever in it: the rows
    from it on are NaN in its elements, the others are as they were."""
    for at in list(range(0, keys, 23)) + [keys // 2, keys - 1]:
        ctx = 2 * keys + at - rows // 2
        c = make([rows], [ctx], 8, 2, D, 16, cache, seed=34)
        clean = run(c, cache)
        poison(c, "vc", 0, [2 * keys + at], NAN, slice(0, None, 5))
        got = run(c, cache)
        sees = torch.arange(c["cap"]) >= rows // 2
        sees[rows:] = False
        assert bool(got[sees][:, :, ::5].isnan().all()), at
        got[sees] = torch.where(got[sees].isnan(), clean[sees], got[sees])
        assert torch.equal(got, clean), at


@pytest.mark.parametrize("D", [64, 128, 96, 136, 192])
@pytest.mark.parametrize("rows,ctx", [([1], [4000]), ([17, 1], [300, 5]), ([150], [40])])
def test_scores_of_minus_infinity_weigh_nothing(D, rows, ctx):
    """Against a key so low that its weight is 0 in 64 bits (exp(-250)) and, where
    every position scores -inf, against zeros."""
    c = make(rows, ctx, 8, 2, D, 16, seed=35)
    c["q"][:, :, 7] = 1.0
    hit = [t for t in range(ctx[0] + rows[0]) if t % 3 == 1]
    poison(c, "kc", 0, hit, -4000.0, slice(7, 8))
    out = torch.zeros((c["cap"], 8, D), dtype=torch.bfloat16)
    want, tol = ref.attend(c["q"], c["kc"], c["vc"], c["cu"], c["ctx"], c["table"],
                           c["max_rows"], out=out)
    poison(c, "kc", 0, hit, -INF, slice(7, 8))
    got = run(c, "bf16").double()
    assert bool(((got - want).abs() <= tol).all())
    poison(c, "kc", 0, range(ctx[0] + rows[0]), -INF, slice(7, 8))
    got = run(c, "bf16").double()
    assert float(got[:rows[0]].abs().max()) == 0.0
    assert bool(((got - want).abs() <= tol)[rows[0]:].all())
