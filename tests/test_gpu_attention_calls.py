"""Attention as callers size and place it: workspaces of the documented size, far
positions (needs an MI355X)."""
import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
import forward_ref as ref
from test_gpu_attention import DEV, SCALES, call, make, pools

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,most", [(32, 40), (1, 33), (17, 4096)])
def test_a_workspace_made_for_more_rows(rows, most):
    """The last, short chunk of a prompt with the workspace of the others."""
    c = make([rows], [700], 32, 8, 128, 16, seed=40)
    c["q"], c["cap"], c["max_rows"] = c["q"][:rows], rows, most
    ws = torch.zeros(dspark.dspark_attention_workspace_bytes(1, most, 32, 8, 128),
                     dtype=torch.uint8, device=DEV)
    out = torch.zeros((rows, 32, 128), dtype=torch.bfloat16)
    want, tol = ref.attend(c["q"], c["kc"], c["vc"], c["cu"], c["ctx"], c["table"], most, out=out)
    kc, vc = pools(c, DEV)
    got = out.to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q, cu, ctx, table = c["q"].to(DEV), i32(c["cu"]), i32(c["ctx"]), c["table"].to(DEV)
    status = dspark.lib().dspark_verify_attention(
        q.data_ptr(), q.stride(0), q.stride(1), kc.data_ptr(), vc.data_ptr(), 0, kc.shape[0], 16,
        *kc.stride()[:3], 1.0, 1.0, table.data_ptr(),
        table.shape[1], cu.data_ptr(), ctx.data_ptr(), 1, rows, most, 32, 8, 128, 0, 128 ** -0.5,
        got.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0
    assert bool(((got.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "e4m3"), (136, "bf16")])
@pytest.mark.parametrize("rows", [3, 150])
@pytest.mark.parametrize("ctx", [2 ** 30 - 70, 2 ** 30 + 5, 1600000000, 2 ** 31 - 2 ** 25 - 1])
def test_positions_past_30_bits(D, cache, rows, ctx):
    """A window at the end of a very long context whose earlier pages are gone: as
    at its start, with the table moved along."""
    page, window = 1024, 200
    base = ctx // page - 1                       # pages before those that matter
    c = make([rows], [ctx - base * page], 4, 2, D, page, cache, seed=41)
    scales = SCALES[cache]
    out = torch.zeros((c["cap"], 4, D), dtype=torch.bfloat16)
    want, tol = ref.attend(c["q"], c["kc"], c["vc"], c["cu"], c["ctx"], c["table"], rows, window,
                           out=out, **scales)
    c["table"] = torch.cat([torch.full((1, base), -1, dtype=torch.int32), c["table"]], 1)
    c["ctx"] = [ctx]
    got = call(c, *pools(c, DEV), out.to(DEV), window=window, **scales)
    torch.cuda.synchronize()
    assert bool(((got.cpu().double() - want).abs() <= tol).all())
