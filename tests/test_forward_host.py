"""Host-side refusals of the operators around the verify forward: every status
comes back before a device is touched, and the binding refuses CPU tensors."""
import ctypes
import os

import pytest
import torch

import __graft_entry__
import confidence_scheduled_ragged_amd as dspark

OK, ENULL, ESHAPE, EARG, EALIGN, EWS, EHIP = range(7)
A = 0x10000          # a fake, 256-byte aligned "device" address; never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dspark.LIB_PATH):
        __graft_entry__.build()
    return dspark.lib()


def ptr(x):
    return ctypes.c_void_p(x) if x else None


def append_call(L, q=A, k=A, v=A, qs=4096, ks=1024, vs=1024, cos=A, sin=A, positions=100, half=64,
                inter=0, cu=A, ctx=A, B=4, rows=8, Hq=32, Hkv=8, D=128, kc=A, vc=A, kind=0,
                pages=10, page=16, ps=16384, hs=2048, ss=128, k_scale=1.0, v_scale=1.0, table=A,
                width=5, out=A):
    return L.dspark_append_kv(ptr(q), ptr(k), ptr(v), qs, ks, vs, ptr(cos), ptr(sin), positions,
                              half, inter, ptr(cu), ptr(ctx), B, rows, Hq, Hkv, D, ptr(kc),
                              ptr(vc), kind, pages, page, ps, hs, ss, k_scale, v_scale, ptr(table),
                              width, ptr(out), None)


SHARED = [(dict(kc=0), ENULL), (dict(vc=0), ENULL), (dict(table=0), ENULL), (dict(cu=0), ENULL),
          (dict(ctx=0), ENULL), (dict(out=0), ENULL), (dict(q=0), ENULL),
          (dict(B=0), ESHAPE), (dict(rows=0), ESHAPE), (dict(rows=(1 << 24) + 1), ESHAPE),
          (dict(Hkv=0), ESHAPE), (dict(Hq=7), ESHAPE), (dict(Hq=4), ESHAPE), (dict(D=0), ESHAPE),
          (dict(pages=0), ESHAPE), (dict(page=0), ESHAPE), (dict(width=0), ESHAPE),
          (dict(page=1 << 20, width=1 << 12), ESHAPE),
          (dict(kind=2), EARG), (dict(kind=-1), EARG), (dict(k_scale=0.0), EARG),
          (dict(v_scale=-1.0), EARG), (dict(k_scale=NAN), EARG), (dict(v_scale=INF), EARG),
          (dict(ps=-8), EARG), (dict(hs=-8), EARG), (dict(ss=-8), EARG),
          (dict(kc=A + 1), EALIGN), (dict(table=A + 2), EALIGN), (dict(cu=A + 1), EALIGN),
          (dict(ctx=A + 2), EALIGN), (dict(q=A + 1), EALIGN), (dict(out=A + 1), EALIGN)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(k=0), ENULL), (dict(cos=0), ENULL), (dict(sin=0), ENULL), (dict(D=1025), ESHAPE),
    (dict(half=65), ESHAPE), (dict(half=-1), ESHAPE), (dict(positions=0), ESHAPE),
    (dict(qs=-1), EARG), (dict(vs=-8), EARG), (dict(cos=A + 2), EALIGN), (dict(v=A + 1), EALIGN)])
def test_append_refusals(L, kw, status):
    assert append_call(L, **kw) == status


def attend_call(L, q=A, qr=4096, qh=128, kc=A, vc=A, kind=0, pages=10, page=16, ps=16384, hs=2048,
                ss=128, k_scale=1.0, v_scale=1.0, table=A, width=5, cu=A, ctx=A, B=4, rows=8,
                max_rows=4, Hq=32, Hkv=8, D=128, window=0, scale=0.1, out=A, ws=A, wsb=1 << 40):
    return L.dspark_verify_attention(ptr(q), qr, qh, ptr(kc), ptr(vc), kind, pages, page, ps, hs,
                                     ss, k_scale, v_scale, ptr(table), width, ptr(cu), ptr(ctx), B,
                                     rows, max_rows, Hq, Hkv, D, window, scale, ptr(out), ptr(ws),
                                     wsb, None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(ws=0), ENULL), (dict(D=264), ESHAPE), (dict(D=12), ESHAPE), (dict(max_rows=0), ESHAPE),
    (dict(window=-1), EARG), (dict(scale=NAN), EARG), (dict(qr=-8), EARG), (dict(qh=-8), EARG),
    (dict(q=A + 8), EALIGN), (dict(out=A + 8), EALIGN), (dict(ws=A + 8), EALIGN),
    (dict(kc=A + 8), EALIGN), (dict(kc=A + 4, kind=1), EALIGN), (dict(ss=132), EALIGN),
    (dict(qr=4100), EALIGN), (dict(wsb=0), EWS)])
def test_attention_refusals(L, kw, status):
    assert attend_call(L, **kw) == status


def test_attention_workspace_bytes(L):
    f = L.dspark_attention_workspace_bytes
    assert f(0, 1, 8, 2, 128) == 0 and f(1, 0, 8, 2, 128) == 0
    assert f(1, 1, 8, 3, 128) == 0 and f(1, 1, 8, 2, 12) == 0 and f(1, 1, 8, 2, 512) == 0
    n = f(4, 17, 32, 8, 128)
    assert n > 0 and n % 256 == 0
    assert attend_call(L, max_rows=4, wsb=f(4, 4, 32, 8, 128) - 1) == EWS


def sample_call(L, logits=A, psrc=A, cu=A, tok=A, u=A, t=A, k=A, p=A, m=A, B=4, g=8, V=1000, smp=A,
                acc=A, bonus=A, ws=A, wsb=1 << 40):
    return L.dspark_sample_accept(ptr(logits), ptr(psrc), ptr(cu), ptr(tok), ptr(u), ptr(t),
                                  ptr(k), ptr(p), ptr(m), B, g, V, ptr(smp), ptr(acc), ptr(bonus),
                                  ptr(ws), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=0), ENULL), (dict(cu=0), ENULL), (dict(tok=0), ENULL), (dict(u=0), ENULL),
    (dict(smp=0), ENULL), (dict(acc=0), ENULL), (dict(bonus=0), ENULL), (dict(ws=0), ENULL),
    (dict(B=0), ESHAPE), (dict(g=0), ESHAPE), (dict(g=257), ESHAPE), (dict(V=0), ESHAPE),
    (dict(B=1 << 24), ESHAPE), (dict(logits=A + 1), EALIGN), (dict(psrc=A + 2), EALIGN),
    (dict(u=A + 2), EALIGN), (dict(t=A + 1), EALIGN), (dict(k=A + 2), EALIGN),
    (dict(p=A + 2), EALIGN), (dict(m=A + 2), EALIGN), (dict(smp=A + 2), EALIGN),
    (dict(ws=A + 8), EALIGN), (dict(wsb=100), EWS)])
def test_sample_refusals(L, kw, status):
    assert sample_call(L, **kw) == status


def test_binding_refuses_cpu_tensors_and_bad_layouts():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    cache = bf(4, 2, 16, 64)
    with pytest.raises(ValueError):
        dspark.dspark_append_kv(bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), torch.zeros(9, 32),
                                torch.zeros(9, 32), i32(2), i32(1), i32(1, 4), cache, cache)
    with pytest.raises(ValueError):
        dspark.dspark_verify_attention(bf(3, 4, 64), cache, cache, i32(2), i32(1), i32(1, 4), 1)
    with pytest.raises(ValueError):
        dspark.dspark_verify_attention(bf(3, 4, 64), cache, cache[:3], i32(2), i32(1), i32(1, 4), 1)
    with pytest.raises(ValueError):
        dspark.dspark_sample_accept(bf(6, 10), None, i32(4), i32(3, 2), torch.zeros(6))


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (8, 8), (64, 8), (40, 8), (9, 1), (127, 1), (128, 1),
                                    (129, 1), (300, 1), (6, 2)])
@pytest.mark.parametrize("D", [64, 72, 128, 136])
def test_attention_workspace_serves_every_smaller_call(L, Hq, Hkv, D):
    """A call has fewer rows than the most its workspace was made for."""
    sizes = [L.dspark_attention_workspace_bytes(1, n, Hq, Hkv, D) for n in range(1, 400)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_attention_accepts_the_workspace_of_its_arguments(L):
    """rows below max_rows: checked against the header's size, one byte below it refused."""
    for rows, most in ((32, 40), (1, 64), (5, 5000)):
        need = L.dspark_attention_workspace_bytes(4, rows, 32, 8, 128)
        assert need <= L.dspark_attention_workspace_bytes(4, most, 32, 8, 128)
        assert attend_call(L, rows=rows, max_rows=most, wsb=need - 1) == EWS


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU, for checks that come before any call."""
    gpu = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.gpu))

    def get_device(self):
        return self.gpu


def on_gpu(x, gpu=0):
    x = x.as_subclass(OnGpu)
    x.gpu = gpu
    return x


def forward_args():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    f32 = torch.zeros
    cache = dict(cu_seqlens=i32(2), ctx_lens=i32(1), block_table=i32(1, 4),
                 k_cache=bf(4, 2, 16, 64), v_cache=bf(4, 2, 16, 64))
    append = dict(q=bf(3, 4, 64), k=bf(3, 2, 64), v=bf(3, 2, 64), cos=f32(9, 32), sin=f32(9, 32),
                  out=bf(3, 4, 64), **cache)
    attend = dict(q=bf(3, 4, 64), max_rows=3, out=bf(3, 4, 64),
                  ws=torch.zeros(1 << 20, dtype=torch.uint8), **cache)
    sample = dict(logits=bf(6, 10), packed_src_row=i32(6), cu_seqlens=i32(4), tokens=i32(3, 2),
                  uniforms=f32(6), temperature=f32(3), top_k=i32(3), top_p=f32(3), min_p=f32(3),
                  packed_sample=i32(6), accepted=i32(3), bonus=i32(3),
                  ws=torch.zeros(1 << 20, dtype=torch.uint8))
    return [(dspark.dspark_append_kv, append), (dspark.dspark_verify_attention, attend),
            (dspark.dspark_sample_accept, sample)]


@pytest.mark.parametrize("i,moved", [(i, k) for i, (_, a) in enumerate(forward_args())
                                     for k, v in a.items() if isinstance(v, torch.Tensor)])
def test_binding_refuses_tensors_on_different_gpus(monkeypatch, i, moved):
    """One tensor on another GPU than all others, whichever it is."""
    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0  # no call reaches a device
    monkeypatch.setattr(dspark, "lib", Lib)
    monkeypatch.setattr(dspark, "_raw_stream", lambda index: 0)
    fn, args = forward_args()[i]

    def call(other):
        a = {k: on_gpu(v, 1 if k == other else 0) if isinstance(v, torch.Tensor) else v
             for k, v in args.items()}
        if fn is dspark.dspark_sample_accept:
            a["out"] = {k: a.pop(k) for k in ("packed_sample", "accepted", "bonus")}
        return fn(**a)
    call(None)
    with pytest.raises(ValueError, match="GPU"):
        call(moved)
