"""Plain 64-bit definitions of the operators around the verify forward, on the
CPU, and the bounds within which a kernel's rounded results must lie."""
import math

import numpy as np
import torch

E4M3_MAX = 448.0
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2      # one rounding, relative
E4M3_HALF = torch.finfo(torch.float8_e4m3fn).eps / 2
E4M3_TINY = 2.0 ** -10                               # half a step below the normal range
F32_HALF = torch.finfo(torch.float32).eps / 2


def slot(table_row, pos, page, pages):
    """(page, slot) of a position, or None where the table names no page."""
    i = pos // page
    if i >= len(table_row) or not 0 <= int(table_row[i]) < pages:
        return None
    return int(table_row[i]), pos % page


def append(q, k, v, cos, sin, cu, ctx, table, k_cache, v_cache, interleaved=False, k_scale=1.0,
           v_scale=1.0, out=None):
    """Float64 results and their error bounds: (out, K, V, out_tol, k_tol); the
    caches [pages, heads, page, D] and `out` in float64, tolerances of what was
    written (0 elsewhere)."""
    e4m3 = k_cache.dtype == torch.float8_e4m3fn
    ks, vs = (k_scale, v_scale) if e4m3 else (1.0, 1.0)
    K, V = k_cache.double(), v_cache.double()
    O = out.double().clone()
    kt, vt, ot = torch.zeros_like(K), torch.zeros_like(V), torch.zeros_like(O)
    half, D = cos.shape[1], q.shape[2]
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)

    def turn(x, p):
        c, s = cos[p].double(), sin[p].double()
        y, mag = x.clone(), x.abs()
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
        mag[:, a] = (x[:, a] * c).abs() + (x[:, b] * s).abs()
        mag[:, b] = (x[:, b] * c).abs() + (x[:, a] * s).abs()
        return y, 3 * F32_HALF * mag

    def store(y, err, scale):
        if not e4m3:
            return y, err + BF16_HALF * y.abs() + 1e-38
        z = (y / scale).clamp(-E4M3_MAX, E4M3_MAX)
        return z, (err + 2 * F32_HALF * y.abs()) / scale + E4M3_HALF * z.abs() + E4M3_TINY

    for n in range(len(ctx)):
        for j in range(cu[n + 1] - cu[n]):
            r, p = cu[n] + j, max(0, ctx[n]) + j
            if r >= q.shape[0] or p >= cos.shape[0]:
                continue
            y, err = turn(q[r].double(), p)
            O[r], ot[r] = y, err + BF16_HALF * y.abs() + 1e-38
            at = slot(table[n], p, k_cache.shape[2], k_cache.shape[0])
            if at is None:
                continue
            y, err = turn(k[r].double(), p)
            K[at[0], :, at[1]], kt[at[0], :, at[1]] = store(y, err, ks)
            y = v[r].double()
            V[at[0], :, at[1]], vt[at[0], :, at[1]] = store(y, torch.zeros_like(y), vs)
    return O, K, V, ot, kt, vt


def attend(q, k_cache, v_cache, cu, ctx, table, max_rows, window=0, scale=None, k_scale=1.0,
           v_scale=1.0, out=None):
    """(out, bound) in float64. The bound counts one bf16 rounding of the result,
    one of every weight before its product with V (2^-8 of the mean of |V|), the
    fp32 dot products (D terms each) and the fp32 sums over the keys."""
    rows, Hq, D = q.shape
    pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    e4m3 = k_cache.dtype == torch.float8_e4m3fn
    ks, vs = (k_scale, v_scale) if e4m3 else (1.0, 1.0)
    scale = D ** -0.5 if scale is None else scale
    O, tol = out.double().clone(), torch.zeros(out.shape, dtype=torch.float64)
    for n in range(len(ctx)):
        c0, count = max(0, ctx[n]), min(max_rows, cu[n + 1] - cu[n])
        top = c0 + count
        at = [slot(table[n], t, page, pages) for t in range(top)]
        pos = torch.tensor([t for t in range(top) if at[t] is not None], dtype=torch.long)
        pg = torch.tensor([at[t][0] for t in pos.tolist()], dtype=torch.long)
        sl = torch.tensor([at[t][1] for t in pos.tolist()], dtype=torch.long)
        K = k_cache[pg, :, sl].double() * ks if len(pos) else torch.zeros(0, Hkv, D).double()
        V = v_cache[pg, :, sl].double() * vs if len(pos) else torch.zeros(0, Hkv, D).double()
        for j in range(count):
            r, p = cu[n] + j, c0 + j
            if r >= rows:
                continue
            see = pos <= p
            if window:
                see &= pos > p - window
            if not bool(see.any()):
                O[r] = 0
                continue
            for h in range(Hq):
                kk, vv = K[see, h // G], V[see, h // G]
                qq = q[r, h].double()
                x = scale * (kk @ qq)
                w = torch.exp(x - x.max())
                w = w / w.sum()
                o = w @ vv
                mean = w @ vv.abs()
                e = 2 * D * F32_HALF * abs(scale) * float((kk.abs() @ qq.abs()).max())
                O[r, h] = o
                tol[r, h] = (BF16_HALF * o.abs()
                             + (BF16_HALF + 2 * e + kk.shape[0] * F32_HALF + 2.0 ** -16) * mean
                             + 1e-30)
    return O, tol


def sample_row(x, u, T, k, p, low):
    """The drawn index of one row of float64 logits."""
    x = np.asarray(x, dtype=np.float64)
    seen = np.nonzero(~np.isnan(x) & (x != -math.inf))[0]
    if seen.size == 0:
        return 0
    order = seen[np.argsort(-x[seen], kind="stable")]
    v = x[order]
    if not T > 0:
        return int(order[0])
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(v == v[0], 1.0, np.exp((v - v[0]) / np.float64(T)))
    n = len(order)
    if k > 0:
        n = min(n, k)
    if p < 1:
        run = np.cumsum(w[:n])
        n = max(1, int(((run - w[:n]) < p * run[-1]).sum()))
    if low > 0:
        n = max(1, int((w[:n] >= low).sum()))
    run = np.cumsum(w[:n])
    return int(order[min(int((run <= max(u, 0.0) * run[-1]).sum()), n - 1)])


def sample_accept(logits, psrc, cu, tokens, uniforms, temperature=None, top_k=None, top_p=None,
                  min_p=None, fill=-1):
    B, W = tokens.shape
    out = np.full(B * W, fill, np.int64)
    acc, bonus = np.zeros(B, np.int64), np.full(B, -1, np.int64)
    for b in range(B):
        for r in range(cu[b], cu[b + 1]):
            src = r if psrc is None else int(psrc[r])
            if not 0 <= src < B * W:
                out[r] = -1
                continue
            out[r] = sample_row(logits[src], float(uniforms[r]),
                                1.0 if temperature is None else float(temperature[b]),
                                0 if top_k is None else int(top_k[b]),
                                1.0 if top_p is None else float(top_p[b]),
                                0.0 if min_p is None else float(min_p[b]))
        n = cu[b + 1] - cu[b]
        a = 0
        while a < n - 1 and out[cu[b] + a] == tokens[b, a + 1]:
            a += 1
        if n > 0:
            acc[b], bonus[b] = a, out[cu[b] + a]
    return out, acc, bonus
