"""What is measured of the operators around the target's verify forward.

Three operators, as a serving loop calls them once per layer or once per step:

* append: rotate the queries and keys of the packed rows by their positions and
  write keys and values into the paged cache (``dspark_append_kv``);
* attend: attention of the packed rows over each request's pages, causal at the
  end of the request (``dspark_verify_attention``): a single new token, a ragged
  verify window, or a whole prompt chunk per request;
* sample: draw the target's token of every packed row (temperature, top-k,
  top-p, min-p, given uniform numbers) and accept the drafts that agree
  (``dspark_sample_accept``).

``run`` computes them in elementary torch operations, or, where ``own`` is true,
through the framework's entry points. ``exact`` writes their definitions out in
64 bits. Sequence lengths, windows and sampling parameters belong to the case
(drawn from its ``mix``); the values in the tensors come from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
E4M3_MAX = 448.0


# --------------------------------------------------------------------- cases

def _append(name, **kw):
    case = dict(name=name, op="append", B=1, gamma=16, rows="single", Hq=32, Hkv=8, D=128, page=64,
                ctx_lo=64, ctx_hi=4096, cache="bf16", rot=128, interleaved=False, mix=1)
    case.update(kw)
    return case


def _attend(name, **kw):
    case = dict(name=name, op="attend", B=1, gamma=16, rows="single", Hq=32, Hkv=8, D=128, page=64,
                ctx_lo=64, ctx_hi=4096, cache="bf16", window=0, mix=1)
    case.update(kw)
    return case


def _sample(name, **kw):
    case = dict(name=name, op="sample", B=1, gamma=16, V=151936, dense=False, filters="mixed", mix=1)
    case.update(kw)
    return case


def listed():
    return [
        # one user, plain decode: one row; launch latency is what counts
        _append("append_single", page=16, ctx_lo=1000, ctx_hi=1000),
        # a full batch of ragged verify windows, the per-layer call of mixed traffic
        _append("append_mixed", B=256, rows="verify", ctx_lo=128, ctx_hi=4096, mix=2),
        # four prompts entering an 8-bit cache, half of each head rotated in pairs
        _append("append_prompt_e4m3", B=4, rows="prompt", gamma=4095, Hq=16, Hkv=4, page=32,
                ctx_lo=0, ctx_hi=0, cache="e4m3", rot=64, interleaved=True, mix=3),
        # one user, one token, an ordinary context: latency and the split over its length
        _attend("attend_single", ctx_lo=4000, ctx_hi=4000, page=16, mix=4),
        # four long documents, short verify windows, an 8-bit cache
        _attend("attend_long_e4m3", B=4, gamma=8, rows="verify", ctx_lo=40000, ctx_hi=120000,
                cache="e4m3", mix=5),
        # the mixed traffic of a full batch: ragged windows, ragged contexts
        _attend("attend_mixed", B=256, rows="verify", ctx_lo=128, ctx_hi=4096, mix=6),
        # sliding-window layer of a model with small heads and a group of five
        _attend("attend_sliding", B=64, rows="verify", Hq=40, Hkv=8, D=64, page=32, ctx_lo=500,
                ctx_hi=12000, window=1024, mix=7),
        # prompts of different lengths packed together, nothing cached before them
        _attend("attend_prompts", B=4, gamma=4095, rows="prompt", ctx_lo=0, ctx_hi=0, mix=8),
        # one chunk of a long prompt on what is cached of it, groups of eight
        _attend("attend_chunk", B=1, gamma=2047, rows="full", Hq=32, Hkv=4, ctx_lo=14000,
                ctx_hi=14000, mix=9),
        # one user's verify block
        _sample("sample_single", mix=10),
        # a small vocabulary and batch, logits left in the dense block
        _sample("sample_tiny_dense", B=4, gamma=8, V=1024, dense=True, mix=11),
        # the full batch of mixed traffic: every request its own parameters
        _sample("sample_mixed", B=256, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    kind = rng.choice(("append", "append_prompt", "attend", "attend", "attend_prompt", "sample"))
    heads = dict(Hkv=rng.choice((1, 2, 3, 4, 8)), D=rng.choice((64, 128, 128)),
                 page=rng.choice((16, 32, 64, 128)), cache=rng.choice(("bf16", "bf16", "e4m3")))
    heads["Hq"] = heads["Hkv"] * rng.choice((1, 2, 3, 4, 5, 8))
    if kind == "append" or kind == "append_prompt":
        rot = rng.choice((heads["D"], heads["D"] // 2))
        more = dict(rot=rot, interleaved=rng.random() < 0.5, mix=mix, **heads)
        if kind == "append":
            return _append("", B=_log_int(rng, 1, 256), gamma=rng.randint(1, 16), ctx_lo=1,
                           ctx_hi=_log_int(rng, 64, 8000), rows=rng.choice(("single", "verify")),
                           **more)
        return _append("", B=rng.randint(1, 4), gamma=_log_int(rng, 100, 3000), ctx_lo=0,
                       ctx_hi=rng.choice((0, 500)), rows="prompt", **more)
    if kind == "attend":
        B = _log_int(rng, 1, 256)
        longest = _log_int(rng, 256, min(60000, 400000 // B))
        return _attend("", B=B, gamma=rng.randint(1, 16), ctx_lo=rng.choice((1, longest // 2)),
                       ctx_hi=longest, rows=rng.choice(("single", "verify", "verify")),
                       window=rng.choice((0, 0, rng.randint(1, 2000))), mix=mix, **heads)
    if kind == "attend_prompt":
        return _attend("", B=rng.randint(1, 4), gamma=_log_int(rng, 40, 2500), ctx_lo=0,
                       ctx_hi=rng.choice((0, 300, 6000)), rows=rng.choice(("prompt", "full")),
                       window=rng.choice((0, 0, 0, rng.randint(16, 2000))), mix=mix, **heads)
    V = _log_int(rng, 1000, 151936)
    return _sample("", B=_log_int(rng, 1, 200), gamma=rng.randint(1, 16), V=V,
                   dense=rng.random() < 0.5, filters=rng.choice(("mixed", "mixed", "none", "all")),
                   mix=mix)


# --------------------------------------------------- lengths, tables, inputs

def _lengths(case):
    """(context, rows) of every request: tokens cached before the call, rows of the call."""
    rng = random.Random(case["mix"])
    top = case["gamma"] + 1
    ctx, rows = [], []
    for _ in range(case["B"]):
        lo, hi = case.get("ctx_lo", 0), case.get("ctx_hi", 0)
        ctx.append(lo if hi <= max(lo, 1) else _log_int(rng, max(lo, 1), hi))
        kind = case.get("rows", "verify")
        if kind == "single":
            rows.append(1)
        elif kind == "full":
            rows.append(top)
        elif kind == "prompt":
            rows.append(rng.randint(max(1, top // 3), top))
        elif rng.random() < 0.35:  # a predictable request keeps its whole block
            rows.append(top)
        else:
            rows.append(1 + min(case["gamma"], int(rng.expovariate(1 / 2.5))))
    return ctx, rows


def _max_rows(case):
    return 1 if case.get("rows") == "single" else case["gamma"] + 1


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cu(rows):
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    return _ints(cu)


def _normal(shape, dtype, gen, std=1.0):
    x = torch.empty(shape, dtype=torch.float32 if dtype == torch.float8_e4m3fn else dtype, device=DEV)
    x.normal_(0.0, std, generator=gen)
    return x.clamp_(-E4M3_MAX, E4M3_MAX).to(dtype) if dtype == torch.float8_e4m3fn else x


def _cache_kind(case):
    e4m3 = case["cache"] == "e4m3"
    # scales as a calibration leaves them: the values fill the 8-bit range
    return (torch.float8_e4m3fn, 0.03125, 0.0234375) if e4m3 else (torch.bfloat16, 1.0, 1.0)


def _prepare_paged(case, gen):
    """The paged cache, its block table and the packed batch's lengths."""
    ctx, rows = _lengths(case)
    page, Hkv, D, B = case["page"], case["Hkv"], case["D"], case["B"]
    dtype, k_scale, v_scale = _cache_kind(case)
    need = [-(-(c + n) // page) for c, n in zip(ctx, rows)]
    # while appending, what precedes a request's last pages is a prefix that all share
    shared = [c // page for c in ctx] if case["op"] == "append" else [0] * B
    prefix = max(shared)
    own_pages = [n - s for n, s in zip(need, shared)]
    pages = prefix + sum(own_pages) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    at = torch.full((B, max(need) + 2), -1, dtype=torch.int64)
    used = prefix
    for b in range(B):
        at[b, :shared[b]] = torch.arange(shared[b])
        at[b, shared[b]:need[b]] = torch.arange(used, used + own_pages[b])
        used += own_pages[b]
    at = at.to(DEV)
    table = torch.where(at >= 0, order[at.clamp(min=0)], torch.full_like(at, -1, dtype=torch.int32))
    shape = (pages, Hkv, page, D)
    return dict(op=case["op"], table=table.contiguous(), cu=_cu(rows), ctx=_ints(ctx), pages=pages,
                k_cache=_normal(shape, dtype, gen, 1.0 / k_scale),
                v_cache=_normal(shape, dtype, gen, 1.0 / v_scale),
                k_scale=k_scale, v_scale=v_scale, max_rows=_max_rows(case),
                longest=max(c + n for c, n in zip(ctx, rows)), capacity=B * _max_rows(case))


def _prepare_append(case, gen):
    s = _prepare_paged(case, gen)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    # queries, keys and values as the fused projection leaves them: one row per token
    s["qkv"] = _normal((s["capacity"], (Hq + 2 * Hkv) * D), torch.bfloat16, gen)
    half = case["rot"] // 2
    angle = (torch.arange(s["longest"], dtype=torch.float64, device=DEV)[:, None]
             * 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half))
    s.update(Hq=Hq, Hkv=Hkv, D=D, cos=angle.cos().float(), sin=angle.sin().float(),
             interleaved=case["interleaved"],
             out=torch.zeros((s["capacity"], Hq, D), dtype=torch.bfloat16, device=DEV))
    return s


def _prepare_attend(case, gen):
    s = _prepare_paged(case, gen)
    shape = (s["capacity"], case["Hq"], case["D"])
    s.update(q=_normal(shape, torch.bfloat16, gen, 1.5), window=case["window"],
             out=torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
    return s


def _prepare_sample(case, gen):
    B, gamma, V = case["B"], case["gamma"], case["V"]
    rng = random.Random(case["mix"] + 1)
    _, rows = _lengths(case)
    logits = _normal((B * (gamma + 1), V), torch.bfloat16, gen, math.sqrt(2.0))
    tokens = torch.randint(0, V, (B, gamma + 1), generator=gen, device=DEV).to(torch.int32)
    # the target mostly agrees with the drafter: a draft's logit stands out at its row
    src = torch.tensor([b * (gamma + 1) + j for b in range(B) for j in range(rows[b])],
                       dtype=torch.int64, device=DEV)
    at = src if case["dense"] else torch.arange(src.numel(), device=DEV)
    draft = torch.cat([tokens[:, 1:], tokens[:, :1]], 1).reshape(-1)[src].long()
    peak = logits[at].amax(1).float() + torch.where(
        torch.rand(src.numel(), generator=gen, device=DEV) < 0.7, 4.0, -4.0)
    logits[at, draft] = peak.to(torch.bfloat16)
    psrc = torch.full((B * (gamma + 1),), -1, dtype=torch.int32, device=DEV)
    psrc[:src.numel()] = src.to(torch.int32)
    pick = lambda mixed, none, all_: {"mixed": mixed, "none": none, "all": all_}[case["filters"]]  # noqa: E731
    f = lambda v: torch.tensor(v, dtype=torch.float32, device=DEV)  # noqa: E731
    temperature = [rng.choice(pick((0.0, 0.6, 0.8, 1.0, 1.3), (1.0,), (0.7, 0.9))) for _ in range(B)]
    top_k = [rng.choice(pick((0, 0, 20, 50, 400), (0,), (40, 64))) for _ in range(B)]
    top_p = [rng.choice(pick((1.0, 0.95, 0.9, 0.6), (1.0,), (0.9, 0.8))) for _ in range(B)]
    min_p = [rng.choice(pick((0.0, 0.0, 0.02, 0.1), (0.0,), (0.01, 0.05))) for _ in range(B)]
    return dict(op="sample", logits=logits, psrc=psrc if case["dense"] else None, cu=_cu(rows),
                tokens=tokens, temperature=f(temperature), top_k=_ints(top_k), top_p=f(top_p),
                min_p=f(min_p),
                uniforms=torch.rand(B * (gamma + 1), generator=gen, device=DEV),
                out=torch.full((B * (gamma + 1),), -1, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + case["mix"])
    return {"append": _prepare_append, "attend": _prepare_attend,
            "sample": _prepare_sample}[case["op"]](case, gen)


# ------------------------------------------------------------------- the work

def work(case):
    ctx, rows = _lengths(case)
    total = sum(rows)
    if case["op"] == "sample":
        return {"bytes": total * (case["V"] * 2 + 12) + case["B"] * 24, "flops": total * case["V"]}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    item = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        moved = total * ((2 * Hq + 2 * Hkv) * D * 2 + 2 * Hkv * D * item + case["rot"] * 4 + 4)
        return {"bytes": moved, "flops": total * (Hq + Hkv) * case["rot"] * 3}
    window = case["window"] or 1 << 40
    kept = pairs = 0
    for c, n in zip(ctx, rows):
        kept += c + n - max(0, c + 1 - window)
        full = max(0, min(n, window - c))  # rows that still see everything before them
        pairs += full * c + full * (full + 1) // 2 + (n - full) * min(window, c + n)
    return {"bytes": kept * Hkv * D * 2 * item + 2 * total * Hq * D * 2 + sum(
                -(-(c + n) // case["page"]) for c, n in zip(ctx, rows)) * 4,
            "flops": pairs * Hq * D * 4}


# ------------------------------------------------------------ the plain forms

def _rows_of(s, capacity):
    """(request, place in its window, whether it is a row) of every packed row."""
    r = torch.arange(capacity, device=DEV)
    total = s["cu"][-1]
    r = torch.minimum(r, total - 1).long()
    b = torch.searchsorted(s["cu"], r.to(torch.int32), right=True) - 1
    return r, b, r - s["cu"].long()[b], torch.arange(capacity, device=DEV) < total


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    part, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([part, rest], -1)


def _raw(cache):
    return cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache


def _stored(x, scale, dtype):
    if dtype == torch.float8_e4m3fn:
        return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(dtype).view(torch.uint8)
    return x.to(dtype)


def _plain_append(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    r, b, j, live = _rows_of(s, s["qkv"].shape[0])
    x = s["qkv"][r].float()
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:]
    pos = s["ctx"].long()[b] + j
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _rotate(q.view(-1, Hq, D), cos, sin, s["interleaved"]).to(torch.bfloat16)
    k = _rotate(k.reshape(-1, Hkv, D), cos, sin, s["interleaved"])
    page = s["k_cache"].shape[2]
    at, off = s["table"][b, pos // page].long(), pos % page
    _raw(s["k_cache"])[at, :, off] = _stored(k, s["k_scale"], s["k_cache"].dtype)
    _raw(s["v_cache"])[at, :, off] = _stored(v.reshape(-1, Hkv, D), s["v_scale"], s["v_cache"].dtype)
    s["out"].copy_(torch.where(live[:, None, None], q, s["out"]))
    return s["out"], s["k_cache"], s["v_cache"]


def _gathered(cache, table, pos):
    """The cache's rows at `pos` of every request, [B, Hkv, len, D] in 32 bits."""
    page = cache.shape[2]
    x = _raw(cache)[table[:, pos // page].long().clamp(min=0), :, (pos % page).expand(table.shape[0], -1)]
    return x.view(cache.dtype).float().transpose(1, 2)


def _plain_attend(s):
    q, cu, ctx = s["q"], s["cu"].long(), s["ctx"].long()
    Hq, D, Hkv, W = q.shape[1], q.shape[2], s["k_cache"].shape[1], s["max_rows"]
    B, G = ctx.numel(), Hq // Hkv
    j = torch.arange(W, device=DEV)
    pos = torch.arange(s["longest"], device=DEV)
    wide = q[(cu[:-1, None] + j).clamp(max=q.shape[0] - 1)].float()
    wide = wide.view(B, W, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * G, D)
    k = _gathered(s["k_cache"], s["table"], pos)
    score = torch.matmul(wide, k.transpose(2, 3)).mul_(s["k_scale"] / math.sqrt(D))
    at = ctx[:, None] + j
    seen = pos <= at[:, :, None]
    if s["window"]:
        seen &= pos > at[:, :, None] - s["window"]
    score = score.view(B, Hkv, W, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["table"], pos)
    o = torch.matmul(p.view(B, Hkv, W * G, -1), v).view(B, Hkv, W, G, D).mul_(s["v_scale"]) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(B, W, Hq, D)
    _, b, place, live = _rows_of(s, q.shape[0])
    s["out"].copy_(torch.where(live[:, None, None], o[b, place].to(q.dtype), s["out"]))
    return s["out"]


def _plain_sample(s):
    logits, cu, tokens = s["logits"], s["cu"].long(), s["tokens"]
    V, B, W = logits.shape[1], tokens.shape[0], tokens.shape[1]
    r, b, j, live = _rows_of(s, logits.shape[0])
    x = logits[s["psrc"].long()[r].clamp(min=0)] if s["psrc"] is not None else logits
    value, index = torch.sort(x.float(), dim=1, descending=True, stable=True)
    value = value.double()
    t = s["temperature"].double()[b, None]
    w = ((value - value[:, :1]) / torch.where(t > 0, t, torch.ones_like(t))).exp_()
    del value
    k = torch.where(t[:, 0] > 0, s["top_k"].long()[b], torch.ones_like(b))[:, None]
    w = torch.where((torch.arange(V, device=DEV) < k) | (k <= 0), w, 0.0)
    run_ = w.cumsum(1)
    p = s["top_p"].double()[b, None]
    w = torch.where((run_ - w < p * run_[:, -1:]) | (p >= 1), w, 0.0)
    w = torch.where(w >= s["min_p"].double()[b, None], w, 0.0)
    run_ = w.cumsum(1)
    rank = (run_ <= s["uniforms"].double()[r, None] * run_[:, -1:]).sum(1, keepdim=True)
    rank = torch.minimum(rank, (w > 0).sum(1, keepdim=True) - 1)
    chosen = index.gather(1, rank)[:, 0].to(torch.int32)
    s["out"].copy_(torch.where(live, chosen, s["out"]))
    # acceptance: the longest run of drafts that the drawn tokens agree with
    place = torch.arange(W - 1, device=DEV)
    drawn = s["out"][(cu[:-1, None] + place).clamp(max=logits.shape[0] - 1)]
    left = (cu[1:] - cu[:-1] - 1)[:, None]
    accepted = ((drawn == tokens[:, 1:]) & (place < left)).long().cumprod(1).sum(1)
    bonus = s["out"][cu[:-1] + accepted]
    return s["out"], accepted.to(torch.int32), bonus


def run(state):
    s = state
    if own:
        import confidence_scheduled_ragged_amd as dspark
        if s["op"] == "append":
            Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
            q, k, v = s["qkv"].view(-1, Hq + 2 * Hkv, D).split((Hq, Hkv, Hkv), 1)
            q = dspark.dspark_append_kv(
                q, k, v, s["cos"], s["sin"], s["cu"], s["ctx"], s["table"], s["k_cache"],
                s["v_cache"], interleaved=s["interleaved"], k_scale=s["k_scale"],
                v_scale=s["v_scale"], out=s["out"])
            return q, s["k_cache"], s["v_cache"]
        if s["op"] == "attend":
            return dspark.dspark_verify_attention(
                s["q"], s["k_cache"], s["v_cache"], s["cu"], s["ctx"], s["table"], s["max_rows"],
                window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
        return dspark.dspark_sample_accept(
            s["logits"], s["psrc"], s["cu"], s["tokens"], s["uniforms"],
            temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
            out={"packed_sample": s["out"]})
    return {"append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}[s["op"]](s)


# --------------------------------------------------- the definitions, 64 bits

def _exact_append(case, s):
    ctx, rows = _lengths(case)
    Hq, Hkv, D, page, half = s["Hq"], s["Hkv"], s["D"], case["page"], case["rot"] // 2
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    out = s["out"].double()
    pairs = [(2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half) for i in range(half)]
    first, second = (torch.tensor(p, device=DEV) for p in zip(*pairs))
    limit = E4M3_MAX if case["cache"] == "e4m3" else math.inf
    start = 0
    for b in range(case["B"]):
        x = s["qkv"][start:start + rows[b]].double().view(rows[b], Hq + 2 * Hkv, D)
        pos = torch.arange(ctx[b], ctx[b] + rows[b], device=DEV)
        turn = torch.complex(s["cos"].double()[pos], s["sin"].double()[pos])[:, None]
        z = torch.complex(x[:, :Hq + Hkv, first], x[:, :Hq + Hkv, second]) * turn
        y = x.clone()
        y[:, :Hq + Hkv, first], y[:, :Hq + Hkv, second] = z.real, z.imag
        out[start:start + rows[b]] = y[:, :Hq]
        at, off = s["table"][b].long()[pos // page], pos % page
        k_cache[at, :, off] = (y[:, Hq:Hq + Hkv] / s["k_scale"]).clamp(-limit, limit)
        v_cache[at, :, off] = (y[:, Hq + Hkv:] / s["v_scale"]).clamp(-limit, limit)
        start += rows[b]
    return out, k_cache, v_cache


def _exact_attend(case, s):
    """Request by request: every head's scores, their softmax over what a row sees, the mean."""
    ctx, rows = _lengths(case)
    page, D, Hkv = case["page"], case["D"], case["Hkv"]
    out = s["out"].double()
    start = 0
    for b in range(case["B"]):
        c, n = ctx[b], rows[b]
        low = max(0, c + 1 - case["window"]) if case["window"] else 0
        pos = torch.arange(low, c + n, device=DEV)
        pages = s["table"][b].long()[pos // page]
        k = s["k_cache"][pages, :, pos % page].double() * s["k_scale"]
        v = s["v_cache"][pages, :, pos % page].double() * s["v_scale"]
        at = torch.arange(c, c + n, device=DEV)[:, None]
        hidden = pos > at
        if case["window"]:
            hidden |= at - pos >= case["window"]
        q = s["q"][start:start + n].double().view(n, Hkv, -1, D)
        for h in range(Hkv):
            score = torch.tensordot(q[:, h], k[:, h], dims=([2], [1])) / math.sqrt(D)
            share = score.masked_fill(hidden[:, None], -math.inf).softmax(2)
            out[start:start + n].view(n, Hkv, -1, D)[:, h] = torch.tensordot(
                share, v[:, h], dims=([2], [0]))
        start += n
    return out


def _exact_sample(case, s):
    """Row by row: the sorted values, then one cut after the other, then the draw."""
    _, rows = _lengths(case)
    out, accepted, bonus = s["out"].long(), [], []
    V, W, r = case["V"], case["gamma"] + 1, 0
    value_of = {k: s[k].double().tolist() for k in ("temperature", "top_k", "top_p", "min_p", "uniforms")}
    for b in range(case["B"]):
        T, p, low = (value_of[k][b] for k in ("temperature", "top_p", "min_p"))
        k = int(value_of["top_k"][b])
        for j in range(rows[b]):
            x = s["logits"][r if s["psrc"] is None else b * W + j].double()
            order = torch.argsort(-x, stable=True)
            if T <= 0:
                order = order[:1]
            elif k > 0:
                order = order[:k]
            w = torch.exp((x[order] - x.max()) / (T if T > 0 else 1.0))
            if p < 1:
                order = order[:int((torch.cumsum(w, 0) < p * w.sum()).sum()) + 1]
            order = order[torch.exp((x[order] - x.max()) / (T if T > 0 else 1.0)) >= low]
            w = torch.exp((x[order] - x.max()) / (T if T > 0 else 1.0))
            at = int((torch.cumsum(w, 0) <= value_of["uniforms"][r] * w.sum()).sum())
            out[r] = order[min(at, order.numel() - 1)]
            r += 1
        drawn, draft = out[r - rows[b]:r].tolist(), s["tokens"][b, 1:].tolist()
        a = 0
        while a < rows[b] - 1 and drawn[a] == draft[a]:
            a += 1
        accepted.append(a)
        bonus.append(drawn[a])
    return out, torch.tensor(accepted), torch.tensor(bonus)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](case, s)
