"""How the attention of trees and sinks divides its work (needs an MI355X): units of
several tiles, a sink tile below the window's, that are handed out whole, one and two
a workgroup, and their neighbours that the rule for it leaves to be cut. Which of the
two ran shows in the workspace, where only cut units leave partial results."""
import random

import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
import tree_ref as ref
from test_gpu_attention import SCALES, make, pools
from test_gpu_tree_attention import call, tree

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
CUS = 256  # that the cases' numbers of units are made for
CONTROL = 1 << 16  # bytes of a workspace that hold more than all its control words


def handed_out_whole(c, window=0, sinks=0):
    """The kernel's rule: the longest unit times the units of a workgroup is at most 1.3
    times the even division. A unit has a place for each of its tiles and four more."""
    Hkv, item = c["kc"].shape[1], c["kc"].element_size()
    keys = 16384 // ((64 if c["D"] <= 64 else 128) * item)  # positions of a tile
    wide = c["max_rows"] * c["Hq"] // Hkv > 128  # blocks of 256 rows, one workgroup a CU
    wgs, places = CUS if wide else 2 * CUS, []
    for b, ctx in enumerate(c["ctx"]):
        n = c["cu"][b + 1] - c["cu"][b]
        first = max(0, ctx + 1 - window) // keys if window else 0
        tiles = -(-(ctx + n) // keys) - first
        places.append(4 + tiles + min(-(-sinks // keys), first))
        assert n > 0 and tiles > 1
    units = len(places) * Hkv
    return max(places) * -(-units // wgs) * 10 <= -(-sum(places) * Hkv // wgs) * 13


def workspace(c):
    need = dspark.dspark_attention_workspace_bytes(len(c["ctx"]), c["max_rows"], c["Hq"],
                                                   c["kc"].shape[1], c["D"])
    assert need > CONTROL
    return torch.zeros(need, dtype=torch.uint8, device=DEV)


def check(c, whole, **kw):
    """Against the definition; the rule takes the case as is said here, and so does the kernel."""
    view = {k: v for k, v in kw.items() if k in ("window", "sinks")}
    assert handed_out_whole(c, **view) == whole
    kc, vc = pools(c, "cpu")
    out = torch.randn((c["cap"], c["Hq"], c["D"])).bfloat16()
    want, tol = ref.attend(c["q"], kc, vc, c["cu"], c["ctx"], c["table"], c["max_rows"],
                           c.get("depths"), c.get("bits"), out=out, **kw)
    ws = workspace(c)
    got = call(c, *pools(c, DEV), out.to(DEV), ws=ws, **kw)
    torch.cuda.synchronize()
    assert bool(ws[CONTROL:].any()) != whole
    off = (got.cpu().double() - want).abs()
    assert bool((off <= tol).all()), (int((off > tol).sum()), float(off.max()))
    return got


def without(c):
    """The case's rows as a chain."""
    return {k: v for k, v in c.items() if k not in ("bits", "depths", "words")}


@pytest.fixture(autouse=True)
def a_whole_device():
    if torch.cuda.get_device_properties(0).multi_processor_count != CUS:
        pytest.skip("the cases are made for %d compute units" % CUS)


@pytest.mark.parametrize("B,whole", [(64, True), (65, False), (128, True)])
@pytest.mark.parametrize("D,cache,window,sinks,ctx", [
    (64, "bf16", 400, 4, 900), (64, "e4m3", 700, 4, 1500), (128, "bf16", 200, 70, 500),
    (128, "e4m3", 300, 20, 900), (96, "bf16", 150, 64, 300)])
def test_units_of_several_tiles_and_a_sink_tile(B, whole, D, cache, window, sinks, ctx):
    """One and two whole units a workgroup; eight units too many for one."""
    rng = random.Random(B + D)
    kw = dict(window=window, sinks=sinks, **SCALES[cache])
    rows, lens = [rng.randint(1, 3) for _ in range(B)], [ctx + b % 7 for b in range(B)]
    c = tree(make(rows, lens, 16, 8, D, 16, cache, seed=B), B, window, sinks)
    check(c, whole, **kw)
    check(without(c), whole, **kw)


@pytest.mark.parametrize("B,whole", [(64, True), (65, False)])
def test_units_without_a_window(B, whole):
    rng = random.Random(B)
    rows = [rng.randint(1, 12) for _ in range(B)]
    c = tree(make(rows, [650 + b % 40 for b in range(B)], 16, 8, 128, 16, seed=B), B)
    check(c, whole)
    check(without(c), whole)


@pytest.mark.parametrize("B,whole", [(32, True), (33, False), (64, True)])
@pytest.mark.parametrize("D,cache,window,sinks,ctx", [
    (64, "bf16", 400, 4, 900), (128, "e4m3", 300, 20, 900), (128, "bf16", 0, 0, 400)])
def test_units_of_more_than_128_rows(B, whole, D, cache, window, sinks, ctx):
    """One and two a workgroup in blocks of 256 rows; eight too many for one."""
    rng = random.Random(B + D)
    kw = dict(window=window, sinks=sinks, **SCALES[cache])
    rows, lens = [rng.randint(8, 12) for _ in range(B)], [ctx + b % 7 for b in range(B)]
    rows[0] = 33  # of one tree alone, so that the definition is soon computed
    c = tree(make(rows, lens, 32, 8, D, 16, cache, seed=B), B, window, sinks)
    check(c, whole, **kw)
    check(without(c), whole, **kw)


@pytest.mark.parametrize("short,whole", [(0, True), (47, True), (48, False), (60, False)])
def test_units_of_two_lengths_on_both_sides_of_the_limit(short, whole):
    """Units of 10 places and of 6: 10 is up to 1.3 times the mean, and more than that."""
    kw = dict(window=400, sinks=4)
    lens = [200 if b < short else 900 + b % 7 for b in range(64)]
    c = tree(make([2] * 64, lens, 8, 8, 64, 16, seed=short), short, **kw)
    check(c, whole, **kw)
    check(without(c), whole, **kw)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_whole_units_with_pages_that_are_not_named_and_slots_that_none_sees(cache):
    """Holes among the sinks and in the window; NaN in every position between them."""
    window, sinks, ctx = 300, 20, 800
    kw = dict(window=window, sinks=sinks, **SCALES[cache])
    c = tree(make([3] * 64, [ctx + b % 5 for b in range(64)], 16, 8, 64, 16, cache, seed=5), 5,
             window, sinks)
    pages = c["kc"].shape[0]
    c["table"][3, 0] = -1
    c["table"][5, 1] = pages
    c["table"][9, ctx // 16 - 3] = -7
    c["table"][11, (ctx - window) // 16 + 2:(ctx - window) // 16 + 9] = pages + 4
    cases = [c, without(c)]
    clean = [check(x, True, **kw)[:c["cu"][-1]].clone() for x in cases]
    for b in range(64):
        for t in range(sinks, c["ctx"][b] + 1 - window):
            at = int(c["table"][b, t // 16])
            if 0 <= at < pages:
                for x in (c["kc"], c["vc"]):
                    raw = x.view(torch.uint8 if cache == "e4m3" else torch.int16)
                    raw[at, :, t % 16] = 0x7F if cache == "e4m3" else 0x7FC0
    for x, want in zip(cases, clean):
        out = torch.zeros((c["cap"], c["Hq"], 64), dtype=torch.bfloat16, device=DEV)
        got = call(x, *pools(x, DEV), out, ws=workspace(x), **kw)
        assert torch.equal(got[:c["cu"][-1]], want)
