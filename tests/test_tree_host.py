"""Host-side refusals of the operators on drafted trees and shared pages: every
status comes back before a device is touched, and the binding refuses tensors that
are not on one GPU."""
import contextlib
import os

import pytest
import torch

import __graft_entry__
import confidence_scheduled_ragged_amd as dspark
from test_forward_host import (A, EALIGN, EARG, ENULL, ESHAPE, EWS, INF, NAN, SHARED, on_gpu, ptr)

MAX_TREE, MAX_ROWS = 1024, 1 << 24


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dspark.LIB_PATH):
        __graft_entry__.build()
    return dspark.lib()


def masks_call(L, parents=A, cu=A, ctx=A, B=4, rows=80, max_rows=40, window=0, sinks=0, words=2,
               depths=A, masks=A):
    return L.dspark_tree_masks(ptr(parents), ptr(cu), ptr(ctx), B, rows, max_rows, window, sinks,
                               words, ptr(depths), ptr(masks), None)


@pytest.mark.parametrize("kw,status", [
    (dict(parents=0), ENULL), (dict(cu=0), ENULL), (dict(depths=0), ENULL), (dict(masks=0), ENULL),
    (dict(ctx=0, window=3, sinks=1), ENULL), (dict(B=0), ESHAPE), (dict(rows=0), ESHAPE),
    (dict(rows=MAX_ROWS + 1), ESHAPE), (dict(B=MAX_ROWS + 1), ESHAPE), (dict(max_rows=0), ESHAPE),
    (dict(max_rows=MAX_TREE + 1, words=33), ESHAPE), (dict(words=1), ESHAPE), (dict(words=0), ESHAPE),
    (dict(words=33), ESHAPE), (dict(window=-1), EARG), (dict(sinks=-1), EARG),
    (dict(parents=A + 2), EALIGN), (dict(cu=A + 1), EALIGN), (dict(ctx=A + 2), EALIGN),
    (dict(depths=A + 2), EALIGN), (dict(masks=A + 2), EALIGN)])
def test_masks_refusals(L, kw, status):
    assert masks_call(L, **kw) == status


def append_call(L, q=A, k=A, v=A, qs=4096, ks=1024, vs=1024, cos=A, sin=A, positions=100, half=64,
                inter=0, depths=A, cu=A, ctx=A, B=4, rows=8, Hq=32, Hkv=8, D=128, kc=A, vc=A,
                kind=0, pages=10, page=16, ps=16384, hs=2048, ss=128, k_scale=1.0, v_scale=1.0,
                table=A, width=5, out=A):
    return L.dspark_append_tree_kv(ptr(q), ptr(k), ptr(v), qs, ks, vs, ptr(cos), ptr(sin), positions,
                                   half, inter, ptr(depths), ptr(cu), ptr(ctx), B, rows, Hq, Hkv, D,
                                   ptr(kc), ptr(vc), kind, pages, page, ps, hs, ss, k_scale,
                                   v_scale, ptr(table), width, ptr(out), None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(depths=0), ENULL), (dict(depths=A + 2), EALIGN), (dict(k=0), ENULL), (dict(cos=0), ENULL),
    (dict(half=65), ESHAPE), (dict(positions=0), ESHAPE), (dict(D=1025), ESHAPE),
    (dict(qs=-1), EARG), (dict(v=A + 1), EALIGN)])
def test_append_refusals(L, kw, status):
    assert append_call(L, **kw) == status


def attend_call(L, q=A, qr=4096, qh=128, kc=A, vc=A, kind=0, pages=10, page=16, ps=16384, hs=2048,
                ss=128, k_scale=1.0, v_scale=1.0, table=A, width=5, cu=A, ctx=A, B=4, rows=80,
                max_rows=40, Hq=32, Hkv=8, D=128, window=0, sinks=0, depths=A, masks=A, words=2,
                scale=0.1, out=A, ws=A, wsb=1 << 40):
    return L.dspark_tree_attention(ptr(q), qr, qh, ptr(kc), ptr(vc), kind, pages, page, ps, hs, ss,
                                   k_scale, v_scale, ptr(table), width, ptr(cu), ptr(ctx), B, rows,
                                   max_rows, Hq, Hkv, D, window, sinks, ptr(depths), ptr(masks),
                                   words, scale, ptr(out), ptr(ws), wsb, None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(ws=0), ENULL), (dict(depths=0), ENULL), (dict(masks=0), ENULL), (dict(D=264), ESHAPE),
    (dict(D=12), ESHAPE), (dict(max_rows=0), ESHAPE), (dict(words=1), ESHAPE),
    (dict(words=0), ESHAPE), (dict(words=-3), ESHAPE), (dict(words=MAX_ROWS), ESHAPE),
    (dict(rows=1 << 20, max_rows=65), ESHAPE), (dict(window=-1), EARG), (dict(sinks=-1), EARG),
    (dict(window=9, sinks=-4), EARG), (dict(scale=NAN), EARG), (dict(scale=INF), EARG),
    (dict(depths=A + 2), EALIGN), (dict(masks=A + 1), EALIGN), (dict(q=A + 8), EALIGN),
    (dict(kc=A + 8), EALIGN), (dict(ss=132), EALIGN), (dict(wsb=0), EWS)])
def test_attention_refusals(L, kw, status):
    assert attend_call(L, **kw) == status


def test_attention_takes_the_workspace_of_dspark_verify_attention(L):
    need = L.dspark_attention_workspace_bytes(4, 40, 32, 8, 128)
    assert attend_call(L, wsb=need - 1) == EWS
    assert attend_call(L, wsb=need - 1, depths=0, masks=0) == EWS


def accept_call(L, choice=A, tokens=A, parents=A, cu=A, B=4, rows=80, max_rows=40, width=9, acc=A,
                bonus=A, path=A):
    return L.dspark_tree_accept(ptr(choice), ptr(tokens), ptr(parents), ptr(cu), B, rows, max_rows,
                                width, ptr(acc), ptr(bonus), ptr(path), None)


@pytest.mark.parametrize("kw,status", [
    (dict(choice=0), ENULL), (dict(tokens=0), ENULL), (dict(parents=0), ENULL), (dict(cu=0), ENULL),
    (dict(acc=0), ENULL), (dict(bonus=0), ENULL), (dict(path=0), ENULL), (dict(B=0), ESHAPE),
    (dict(rows=0), ESHAPE), (dict(max_rows=0), ESHAPE), (dict(max_rows=MAX_TREE + 1), ESHAPE),
    (dict(width=0), ESHAPE), (dict(width=MAX_TREE + 1), ESHAPE), (dict(choice=A + 2), EALIGN),
    (dict(tokens=A + 1), EALIGN), (dict(parents=A + 2), EALIGN), (dict(cu=A + 2), EALIGN),
    (dict(acc=A + 2), EALIGN), (dict(bonus=A + 2), EALIGN), (dict(path=A + 2), EALIGN)])
def test_accept_refusals(L, kw, status):
    assert accept_call(L, **kw) == status


POOLS = dict(kc=A, vc=A, kind=0, layers=2, ls=1 << 20, pages=10, page=16, ps=16384, hs=2048, ss=128,
             Hkv=8, D=128)
POOL_REFUSALS = [
    (dict(kc=0), ENULL), (dict(vc=0), ENULL), (dict(layers=0), ESHAPE), (dict(layers=32768), ESHAPE),
    (dict(pages=0), ESHAPE), (dict(page=0), ESHAPE), (dict(Hkv=0), ESHAPE), (dict(Hkv=4097), ESHAPE),
    (dict(D=0), ESHAPE), (dict(D=1025), ESHAPE), (dict(kind=2), EARG), (dict(kind=-1), EARG),
    (dict(ls=-1), EARG), (dict(ps=-1), EARG), (dict(hs=-1), EARG), (dict(ss=-1), EARG),
    (dict(kc=A + 1), EALIGN), (dict(vc=A + 1), EALIGN)]


def pool_args(kw):
    p = dict(POOLS, **{k: v for k, v in kw.items() if k in POOLS})
    return [ptr(p.pop("kc")), ptr(p.pop("vc")), *p.values()]


@pytest.mark.parametrize("kw,status", POOL_REFUSALS + [
    (dict(path=0), ENULL), (dict(acc=0), ENULL), (dict(ctx=0), ENULL), (dict(table=0), ENULL),
    (dict(width=0), ESHAPE), (dict(width=MAX_TREE + 1), ESHAPE), (dict(tw=0), ESHAPE),
    (dict(tw=1 << 28), ESHAPE), (dict(B=0), ESHAPE), (dict(B=MAX_ROWS + 1), ESHAPE),
    (dict(path=A + 2), EALIGN), (dict(acc=A + 1), EALIGN), (dict(ctx=A + 2), EALIGN),
    (dict(table=A + 2), EALIGN)])
def test_move_refusals(L, kw, status):
    a = dict(dict(path=A, acc=A, width=9, ctx=A, table=A, tw=5, B=4), **kw)
    assert L.dspark_move_kv(*pool_args(kw), ptr(a["path"]), ptr(a["acc"]), a["width"],
                            ptr(a["ctx"]), ptr(a["table"]), a["tw"], a["B"], None) == status


@pytest.mark.parametrize("kw,status", POOL_REFUSALS + [
    (dict(src=0), ENULL), (dict(dst=0), ENULL), (dict(n=0), ESHAPE), (dict(n=(1 << 20) + 1), ESHAPE),
    (dict(src=A + 2), EALIGN), (dict(dst=A + 2), EALIGN), (dict(slots=A + 1), EALIGN)])
def test_copy_refusals(L, kw, status):
    a = dict(dict(src=A, dst=A, slots=A, n=4), **kw)
    assert L.dspark_copy_pages(*pool_args(kw), ptr(a["src"]), ptr(a["dst"]), ptr(a["slots"]),
                               a["n"], None) == status


TABLE = dict(table=A, held=A, lens=A, R=4, width=9, page=16, refs=A, pages=50)
TABLE_REFUSALS = [
    (dict(table=0), ENULL), (dict(held=0), ENULL), (dict(lens=0), ENULL), (dict(refs=0), ENULL),
    (dict(granted=0), ENULL), (dict(R=0), ESHAPE), (dict(R=(1 << 20) + 1), ESHAPE),
    (dict(width=0), ESHAPE), (dict(page=0), ESHAPE), (dict(pages=0), ESHAPE),
    (dict(pages=(1 << 30) + 1), ESHAPE), (dict(width=1 << 20, page=1 << 11), ESHAPE),
    (dict(R=1 << 20, width=(1 << 10) + 1), ESHAPE),
    (dict(table=A + 2), EALIGN), (dict(held=A + 1), EALIGN), (dict(lens=A + 2), EALIGN),
    (dict(refs=A + 2), EALIGN), (dict(granted=A + 2), EALIGN)]


def table_args(kw):
    p = dict(TABLE, **{k: v for k, v in kw.items() if k in TABLE})
    return [ptr(p[k]) if k in ("table", "held", "lens", "refs") else p[k] for k in TABLE]


@pytest.mark.parametrize("kw,status", TABLE_REFUSALS)
def test_resize_refusals(L, kw, status):
    assert L.dspark_resize_pages(*table_args(kw), ptr(kw.get("granted", A)), None) == status


@pytest.mark.parametrize("kw,status", TABLE_REFUSALS + [
    (dict(src=0), ENULL), (dict(dst=0), ENULL), (dict(cs=0), ENULL), (dict(cd=0), ENULL),
    (dict(ct=0), ENULL), (dict(n=0), ESHAPE), (dict(n=16385), ESHAPE), (dict(src=A + 2), EALIGN),
    (dict(dst=A + 2), EALIGN), (dict(cs=A + 2), EALIGN), (dict(cd=A + 2), EALIGN),
    (dict(ct=A + 2), EALIGN)])
def test_fork_refusals(L, kw, status):
    a = dict(dict(src=A, dst=A, n=3, cs=A, cd=A, ct=A, granted=A), **kw)
    assert L.dspark_fork_pages(*table_args(kw), ptr(a["src"]), ptr(a["dst"]), a["n"], ptr(a["cs"]),
                               ptr(a["cd"]), ptr(a["ct"]), ptr(a["granted"]), None) == status


# -------------------------------------------------------------------- binding

def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def calls():
    """(entry, its tensors by name, other arguments)"""
    paged = dict(cu_seqlens=i32(2), ctx_lens=i32(1), block_table=i32(1, 4),
                 k_cache=bf16(4, 2, 16, 64), v_cache=bf16(4, 2, 16, 64))
    layers = dict(k_cache=bf16(3, 4, 2, 16, 64), v_cache=bf16(3, 4, 2, 16, 64))
    table = dict(table=i32(2, 3), held=i32(2), refs=i32(9), lens=i32(2))
    return [
        (dspark.dspark_tree_masks, dict(parents=i32(3), cu_seqlens=i32(2), ctx_lens=i32(1),
                                        out=(i32(3), i32(3, 1))), dict(max_rows=3)),
        (dspark.dspark_append_tree_kv, dict(q=bf16(3, 4, 64), k=bf16(3, 2, 64), v=bf16(3, 2, 64),
                                            cos=torch.zeros(9, 32), sin=torch.zeros(9, 32),
                                            depths=i32(3), out=bf16(3, 4, 64), **paged), {}),
        (dspark.dspark_tree_attention, dict(q=bf16(3, 4, 64), depths=i32(3), masks=i32(3, 1),
                                            out=bf16(3, 4, 64),
                                            ws=torch.zeros(9, dtype=torch.uint8), **paged),
         dict(max_rows=3)),
        (dspark.dspark_tree_accept, dict(packed_choice=i32(3), packed_tokens=i32(3), parents=i32(3),
                                         cu_seqlens=i32(2), out=(i32(1), i32(1), i32(1, 4))),
         dict(max_rows=3, width=4)),
        (dspark.dspark_move_kv, dict(path=i32(1, 4), accepted=i32(1), ctx_lens=i32(1),
                                     block_table=i32(1, 4), **layers), {}),
        (dspark.dspark_resize_pages, dict(granted=i32(2), **table), dict(page_size=16)),
        (dspark.dspark_fork_pages, dict(src=i32(1), dst=i32(1), out=(i32(1), i32(1), i32(1), i32(1)),
                                        **table), dict(page_size=16)),
        (dspark.dspark_copy_pages, dict(src=i32(2), dst=i32(2), slots=i32(2), **layers), {}),
    ]


def names(tensors):
    return [(k, i) for k, v in tensors.items()
            for i in (range(len(v)) if isinstance(v, tuple) else [None])]


def placed(tensors, gpu_of):
    return {k: tuple(on_gpu(x, gpu_of(k, i)) for i, x in enumerate(v)) if isinstance(v, tuple)
            else on_gpu(v, gpu_of(k, None)) for k, v in tensors.items()}


@pytest.fixture
def no_device(monkeypatch):
    """Calls end at the library's door; what reached it is noted."""
    reached = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: reached.append((name, a)) or 0
    monkeypatch.setattr(dspark, "lib", Lib)
    monkeypatch.setattr(dspark, "_raw_stream", lambda index: 1000 + index)
    return reached


@pytest.mark.parametrize("i,moved", [(i, m) for i, c in enumerate(calls()) for m in names(c[1])])
def test_binding_refuses_tensors_on_different_gpus(no_device, i, moved):
    fn, tensors, rest = calls()[i]
    fn(**placed(tensors, lambda k, j: 0), **rest)
    assert [name for name, _ in no_device] == [fn.__name__]
    with pytest.raises(ValueError, match="GPU"):
        fn(**placed(tensors, lambda k, j: int((k, j) == moved)), **rest)
    assert len(no_device) == 1


@pytest.mark.parametrize("i", range(len(calls())))
def test_binding_refuses_cpu_tensors(no_device, i):
    fn, tensors, rest = calls()[i]
    with pytest.raises(ValueError):
        fn(**tensors, **rest)
    assert not no_device


@pytest.mark.parametrize("i", range(len(calls())))
def test_calls_run_on_the_gpu_of_their_tensors(no_device, monkeypatch, i):
    """Where it is not the current one, it is made current for the call."""
    within = []

    @contextlib.contextmanager
    def device(gpu):
        within.append(gpu)
        yield
        within.append(None)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "device", device)
    fn, tensors, rest = calls()[i]
    fn(**placed(tensors, lambda k, j: 1), **rest)
    assert within == [1, None]
    assert no_device[0][1][-1] == 1001  # the stream of that GPU


@pytest.mark.parametrize("i,name,bad", [
    (0, "parents", torch.zeros(3)), (0, "parents", i32(3, 2)[:, 0]), (0, "ctx_lens", i32(2)),
    (0, "out", (i32(2), i32(3, 1))), (0, "out", (i32(3), i32(4, 1))), (1, "depths", i32(2)),
    (1, "depths", torch.zeros(3)), (2, "depths", None), (2, "masks", None), (2, "masks", i32(3)),
    (2, "masks", i32(4, 1)), (2, "masks", torch.zeros(3, 1)), (3, "packed_tokens", i32(4)),
    (3, "parents", i32(2)), (3, "out", (i32(1), i32(1), i32(1, 5))), (4, "path", i32(4)),
    (4, "accepted", i32(2)), (4, "block_table", i32(2, 4)), (4, "k_cache", bf16(3, 4, 2, 16, 32)),
    (4, "v_cache", bf16(3, 4, 16, 2, 64).transpose(2, 3)), (5, "held", i32(3)),
    (5, "lens", i32(1)), (5, "refs", torch.zeros(9)), (5, "granted", i32(3)), (6, "dst", i32(2)),
    (6, "out", (i32(1), i32(1), i32(2), i32(1))), (6, "table", i32(2, 3, 1)), (7, "dst", i32(1)),
    (7, "slots", i32(3)), (7, "v_cache", bf16(3, 4, 2, 16, 64).float())])
def test_binding_refuses_other_shapes_and_types(no_device, i, name, bad):
    fn, tensors, rest = calls()[i]
    tensors = dict(tensors, **{name: bad})
    kept = {k: v for k, v in tensors.items() if v is not None}
    with pytest.raises((ValueError, TypeError)):
        fn(**placed(kept, lambda k, j: 0), **rest)
    assert not no_device


def test_masks_with_window_and_sinks_need_the_contexts(no_device):
    with pytest.raises(ValueError, match="ctx_lens"):
        dspark.dspark_tree_masks(on_gpu(i32(3)), on_gpu(i32(2)), 3, window=4, sinks=2)


def test_a_new_pool():
    table, held, refs = dspark.page_pool(7, 3, 5, "cpu")
    assert table.shape == (3, 5) and bool((table == -1).all())
    assert held.shape == (3,) and refs.shape == (7,) and not held.any() and not refs.any()
    assert {t.dtype for t in (table, held, refs)} == {torch.int32}
