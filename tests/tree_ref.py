"""Plain definitions of the operators on drafted trees and shared pages, on the
CPU, and the bounds within which a kernel's rounded results must lie."""
import random

import torch

import forward_ref as ref
from forward_ref import BF16_HALF, F32_HALF, slot


def some_tree(rng, n, branch=0.5):
    """Parents of n nodes: each hangs on an earlier one, the last one more often."""
    return [-1] + [i - 1 if rng.random() > branch else rng.randrange(i) for i in range(1, n)]


def lineage(parents, j):
    """Node j, its parent, and so on up to its root."""
    up = [j]
    while 0 <= parents[up[-1]] < up[-1]:
        up.append(parents[up[-1]])
    return up


def masks(parents, cu, max_rows, words, ctx=None, window=0, sinks=0):
    """{row: (depth, [bits of every word])} of the rows that the call writes."""
    out = {}
    for b in range(len(cu) - 1):
        s, n = cu[b], min(max_rows, cu[b + 1] - cu[b])
        for j in range(n):
            up = lineage(parents[s:s + n], j)
            depth, bits = len(up) - 1, 0
            for step, k in enumerate(up):
                at = (max(0, ctx[b]) if ctx else 0) + depth - step
                if window == 0 or step < window or at < sinks:
                    bits |= 1 << k
            out[s + j] = depth, [bits >> (32 * w) & 0xFFFFFFFF for w in range(words)]
    return out


def signed(word):
    return word - (1 << 32) if word >> 31 else word


def seen(ctx, n, j, depth, bits, window, sinks):
    """Positions that row j of n sees: bits None for a chain, an integer otherwise."""
    if bits is None:
        return [t for t in range(ctx + j + 1) if not window or t > ctx + j - window or t < sinks]
    p = ctx + min(max(depth, 0), j)
    return ([t for t in range(ctx) if not window or t > p - window or t < sinks]
            + [ctx + i for i in range(n) if bits >> i & 1])


def attend(q, k_cache, v_cache, cu, ctx, table, max_rows, depths=None, bits=None, window=0, sinks=0,
           scale=None, k_scale=1.0, v_scale=1.0, out=None):
    """(out, bound) in float64; depths and bits (integers) per packed row. The bound
    counts what forward_ref.attend's does: one bf16 rounding of the result and of every
    weight, the fp32 dot products and the fp32 sums over the keys."""
    rows, Hq, D = q.shape
    pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    e4m3 = k_cache.dtype == torch.float8_e4m3fn
    ks, vs = (k_scale, v_scale) if e4m3 else (1.0, 1.0)
    scale = D ** -0.5 if scale is None else scale
    O, tol = out.double().clone(), torch.zeros(out.shape, dtype=torch.float64)
    for b in range(len(ctx)):
        c, n = max(0, ctx[b]), min(max_rows, cu[b + 1] - cu[b])
        for j in range(n):
            r = cu[b] + j
            if r >= rows:
                continue
            at = [slot(table[b], t, page, pages)
                  for t in seen(c, n, j, None if depths is None else depths[r],
                                None if bits is None else bits[r], window, sinks)]
            at = [a for a in at if a is not None]
            O[r] = 0
            if not at:
                continue
            pg, sl = torch.tensor(at).t()
            K, V = k_cache[pg, :, sl].double() * ks, v_cache[pg, :, sl].double() * vs
            qq = q[r].double().view(Hkv, G, D)
            x = scale * torch.einsum("hgd,nhd->hgn", qq, K)
            w = torch.softmax(x, -1)
            O[r] = torch.einsum("hgn,nhd->hgd", w, V).reshape(Hq, D)
            mean = torch.einsum("hgn,nhd->hgd", w, V.abs()).reshape(Hq, D)
            big = torch.einsum("hgd,nhd->hgn", qq.abs(), K.abs()).amax(-1).reshape(Hq, 1)
            e = 2 * D * F32_HALF * abs(scale) * big
            tol[r] = (BF16_HALF * O[r].abs()
                      + (BF16_HALF + 2 * e + len(at) * F32_HALF + 2.0 ** -16) * mean + 1e-30)
    return O, tol


def append(q, k, v, cos, sin, depths, cu, ctx, table, k_cache, v_cache, **kw):
    """forward_ref.append, a node's angles put where its slot's are looked up: row by
    row, each a request of its own."""
    out = kw.pop("out")
    total = [out.double().clone(), k_cache.double(), v_cache.double()]
    tol = [torch.zeros_like(x) for x in total]
    for b in range(len(ctx)):
        for j in range(cu[b + 1] - cu[b]):
            r = cu[b] + j
            place = max(0, ctx[b]) + j
            pos = max(0, ctx[b]) + min(max(depths[r], 0), j)
            if r >= q.shape[0] or pos >= cos.shape[0]:
                continue
            c = torch.zeros(place + 1, cos.shape[1])
            s = torch.zeros_like(c)
            c[place], s[place] = cos[pos], sin[pos]
            got = ref.append(q[r:r + 1], k[r:r + 1], v[r:r + 1], c, s, [0, 1], [place],
                             table[b:b + 1], k_cache, v_cache, out=out[r:r + 1], **kw)
            total[0][r], tol[0][r] = got[0][0], got[3][0]
            at = slot(table[b], place, k_cache.shape[2], k_cache.shape[0])
            if at is not None:
                for i in (1, 2):
                    total[i][at[0], :, at[1]] = got[i][at[0], :, at[1]]
                    tol[i][at[0], :, at[1]] = got[i + 3][at[0], :, at[1]]
    return total, tol


def accept(choice, tokens, parents, cu, max_rows, width):
    accepted, bonus, paths = [], [], []
    for b in range(len(cu) - 1):
        s, n = cu[b], min(max_rows, cu[b + 1] - cu[b])
        path = [0] if n > 0 else []
        while path and len(path) < width:
            child = [c for c in range(path[-1] + 1, n) if parents[s + c] == path[-1]
                     and tokens[s + c] == choice[s + path[-1]]]
            if not child:
                break
            path.append(child[0])
        accepted.append(max(len(path) - 1, 0))
        bonus.append(choice[s + path[-1]] if path else -1)
        paths.append(path + [-1] * (width - len(path)))
    return accepted, bonus, paths


class Pool:
    """The pages' state in lists; the lowest free page is always the next."""

    def __init__(self, pages, rows, width, page):
        self.refs, self.page, self.width = [0] * pages, page, width
        self.table, self.held = [[-1] * width for _ in range(rows)], [0] * rows

    def _release(self, b, keep):
        while self.held[b] > keep:
            self.held[b] -= 1
            at = self.table[b][self.held[b]]
            if 0 <= at < len(self.refs):
                self.refs[at] -= 1
            self.table[b][self.held[b]] = -1

    def resize(self, lens):
        want = [-(-max(n, 0) // self.page) for n in lens]
        granted = [int(w <= self.width) for w in want]
        for b, w in enumerate(want):
            if granted[b]:
                self._release(b, w)
        short = False
        for b, w in enumerate(want):
            if not granted[b] or self.held[b] >= w:
                continue
            free = [p for p, n in enumerate(self.refs) if n == 0][:w - self.held[b]]
            short |= len(free) < w - self.held[b]
            if short:
                granted[b] = 0
                continue
            for p in free:
                self.refs[p] = 1
                self.table[b][self.held[b]] = p
                self.held[b] += 1
        return granted

    def fork(self, src, dst, lens):
        """Every entry's (copy_src, copy_dst, copy_slots, granted)."""
        R, out, plans = len(self.table), [], []
        free = [p for p, n in enumerate(self.refs) if n == 0]
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < R and 0 <= d < R) or d in src or d in dst[:i]:
                out.append((-1, -1, 0, 0))
                continue
            full, rest = divmod(min(max(lens[s], 0), self.held[s] * self.page), self.page)
            if rest and not free:
                out.append((-1, -1, 0, 0))
                continue
            fresh = free.pop(0) if rest else -1
            part = self.table[s][full] if rest else -1
            ok = 0 <= part < len(self.refs)
            out.append((part if ok else -1, fresh, rest if ok else 0, 1))
            plans.append((s, d, full, fresh))
        for s, d, full, fresh in plans:
            for p in self.table[s][:full]:
                if 0 <= p < len(self.refs):
                    self.refs[p] += 1
        for s, d, full, fresh in plans:
            self._release(d, 0)
            row = self.table[s][:full] + ([fresh] if fresh >= 0 else [])
            if fresh >= 0:
                self.refs[fresh] = 1
            self.table[d][:len(row)] = row
            self.held[d] = len(row)
        return out


def some_lens(seed, rows, hi):
    rng = random.Random(seed)
    return [rng.choice((0, 1, rng.randint(0, hi))) for _ in range(rows)]
