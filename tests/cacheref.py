"""Plain 64-bit definitions of the paged-cache operators (numpy), the inputs
of their tests and the tolerances of attention."""
from __future__ import annotations

import math

import numpy as np
import torch

# half a step of rounding to the type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
F32 = 2.0 ** -24


# ---------------------------------------------------------------------------
# page plan

def plan(ctx, n, N, page, table, held, ring, state, depth=None):
    """Returns the new (table, held, ring, state) and (slot, pos, missing)."""
    table, held, ring = table.copy(), held.copy(), ring.copy()
    width, P = table.shape[1], len(ring)
    head, count = int(state[0]), int(state[1])
    batch = len(ctx)
    need = [-(-(int(ctx[b]) + int(n[b]) + 1) // page) for b in range(batch)]
    gone = []
    for b in range(batch):
        for j in range(min(need[b], width), held[b]):
            gone.append(table[b, j])
            table[b, j] = -1
        held[b] = min(held[b], max(min(need[b], width), 0))
    left, taken = count, 0
    for b in range(batch):
        want = min(need[b], width) - held[b]
        if want > left:
            left = -1  # nobody after this one gets pages
        if want <= 0 or left < 0:
            continue
        for _ in range(want):
            table[b, held[b]] = ring[(head + taken) % P]
            held[b] += 1
            taken += 1
        left -= want
    for i, p in enumerate(gone):
        ring[(head + count + i) % P] = p
    state = np.array([(head + taken) % P, count - taken + len(gone)],
                     np.int32)
    slot = np.full((batch, N + 1), -1, np.int64)
    pos = np.full((batch, N + 1), -1, np.int32)
    for b in range(batch):
        for i in range(int(n[b]) + 1):
            p = int(ctx[b]) + i
            if p // page < held[b]:
                slot[b, i] = int(table[b, p // page]) * page + p % page
            pos[b, i] = ctx[b] + (0 if i == 0 else
                                  (0 if depth is None else depth[b, i - 1]))
    missing = np.array([need[b] - held[b] for b in range(batch)], np.int32)
    return (table, held, ring, state), (slot, pos, missing)


# ---------------------------------------------------------------------------
# trees

def random_trees(rng, batch, N, n):
    """Parents in node order with their depths and ancestry [N][N]."""
    parent = np.full((batch, N), -1, np.int32)
    depth = np.zeros((batch, N), np.int32)
    anc = np.zeros((batch, N, N), bool)
    for b in range(batch):
        for i in range(max(int(n[b]), 0)):
            p = int(rng.integers(-1, i)) if i > 0 else -1
            parent[b, i] = p
            depth[b, i] = 1 + (depth[b, p] if p >= 0 else 0)
            if p >= 0:
                anc[b, i] = anc[b, p]
            anc[b, i, i] = True
    return parent, depth, anc


def pack(anc):
    batch, N, _ = anc.shape
    W = (N + 63) // 64
    bits = np.zeros((batch, N, W * 64), bool)
    bits[:, :, :N] = anc
    return np.packbits(bits, axis=2, bitorder="little").view(np.int64)


# ---------------------------------------------------------------------------
# attention

def attention(q, kc, vc, table, ctx, n, anc, scale, out_type):
    """float64 (out, lse, tol_out, tol_lse); rows past n are NaN.  anc
    [batch][N][N] or None (node i sees nodes 0..i).

    Tolerances.  A score is a sum of D exact products (16-bit factors) with
    fp32 additions, times an fp32 constant: off by at most
    (D + 3) 2^-24 scale sum |q k| =: ds.  A probability is off by a factor
    e^{2 ds} (its score and the maximum's) times the rounding to the type u
    (half a step) and a few fp32 steps; sums of T terms in fp32 add T 2^-24
    each, the split's join some steps more.  With A = softmax . |v| >= |out|:
    |error| <= A (2 u + (e^{2 ds} - 1) + (2 T + 64) 2^-24), of which one u is the
    result's own rounding.  fp16 also loses what lies below its least step
    2^-24: half of that per probability and in the result."""
    batch, R, Hq, D = q.shape
    n_pages, Hkv, page, _ = kc.shape
    G = Hq // Hkv
    cap = table.shape[1] * page
    out = np.full((batch, R, Hq, D), np.nan)
    lse = np.full((batch, R, Hq), np.nan)
    tol = np.zeros((batch, R, Hq, D))
    tol_l = np.zeros((batch, R, Hq))
    u = HALF_STEP[out_type]
    for b in range(batch):
        m = int(n[b]) + 1
        if m <= 0:
            continue
        L = min(int(ctx[b]) + m, cap)
        t = np.arange(L)
        pages = table[b][t // page]
        live = (pages >= 0) & (pages < n_pages)
        see = np.zeros((m, L), bool)
        for i in range(m):
            see[i] = t <= ctx[b]
            node = t - ctx[b] - 1
            on = (node >= 0) & (node < m - 1)
            if i > 0:
                see[i, on] = (anc[b, i - 1, node[on]] if anc is not None
                              else node[on] < i)
        see &= live[None]
        t = t[live]
        see = see[:, live]
        at, off = pages[live], t % page
        for h in range(Hkv):
            K, Vv = kc[at, h, off], vc[at, h, off]  # [len][D]
            for g in range(G):
                hq = h * G + g
                Q = q[b, :m, hq]
                with np.errstate(invalid="ignore", over="ignore"):
                    S = Q @ K.T * scale
                    ds = ((np.abs(Q) @ np.abs(K).T) * abs(scale)
                          * (D + 3) * F32)
                for i in range(m):
                    w = see[i]
                    if not w.any():
                        out[b, i, hq] = 0.0
                        lse[b, i, hq] = -math.inf
                        continue
                    s = S[i, w]
                    with np.errstate(invalid="ignore"):
                        top = s.max()
                        p = np.exp(s - top)
                        tot = p.sum()
                        out[b, i, hq] = (p @ Vv[w]) / tot
                        A = (p @ np.abs(Vv[w])) / tot
                        lse[b, i, hq] = top + math.log(tot)
                        d = ds[i, w].max()
                        T = int(w.sum())
                        e32 = math.expm1(2 * d) + (2 * T + 64) * F32
                        tol[b, i, hq] = A * (2 * u + e32)
                        tol_l[b, i, hq] = d + (2 * T + 64) * F32 + \
                            abs(lse[b, i, hq]) * 8 * F32
                        if out_type == torch.float16:
                            tol[b, i, hq] += 2.0 ** -25 * (
                                1 + T * np.abs(Vv[w]).max())
    return out, lse, tol, tol_l


class Case:
    """Random inputs of an attention call; everything the rows do not see is
    NaN in the caches."""

    def __init__(self, seed, batch, N, Hq, Hkv, D, page, ctx, n=None,
                 chain=False, dtype=torch.bfloat16, drop=0.0, spread=1.0,
                 scale=None, spare=3):
        rng = np.random.default_rng(seed)
        self.rng, self.dtype = rng, dtype
        self.batch, self.N, self.page = batch, N, page
        self.ctx = np.broadcast_to(np.asarray(ctx, np.int64), batch).copy()
        self.n = np.full(batch, N) if n is None else np.asarray(n, np.int64)
        self.scale = D ** -0.5 if scale is None else scale
        need = -(-(self.ctx + self.n + 1) // page)
        width = max(int(need.max()), 1) + 1
        self.n_pages = int(need.sum()) + spare
        perm = rng.permutation(self.n_pages)
        self.table = np.full((batch, width), -1, np.int32)
        at = 0
        for b in range(batch):
            self.table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
        shape = (self.n_pages, Hkv, page, D)
        self.k = torch.full(shape, math.nan, dtype=dtype)
        self.v = torch.full(shape, math.nan, dtype=dtype)
        for b in range(batch):
            t = np.arange(self.ctx[b] + self.n[b] + 1)
            p = torch.from_numpy(self.table[b][t // page].astype(np.int64))
            o = torch.from_numpy(t % page)
            for c, sp in ((self.k, spread), (self.v, 1.0)):
                x = rng.standard_normal((len(t), Hkv, D)) * sp
                c[p, :, o] = torch.from_numpy(x).to(dtype)
        self.q = torch.from_numpy(rng.standard_normal(
            (batch, N + 1, Hq, D))).to(dtype)
        self.parent, self.depth, anc = random_trees(rng, batch, N, self.n)
        self.anc = None if chain or N == 0 else anc
        if drop > 0:  # pages taken away from the table
            gone = rng.random(self.table.shape) < drop
            bad = rng.choice([-1, -7, self.n_pages, 2 ** 30],
                             self.table.shape)
            self.table = np.where(gone, bad, self.table).astype(np.int32)

    def want(self):
        f = lambda x: x.double().numpy()  # noqa: E731
        return attention(f(self.q), f(self.k), f(self.v), self.table,
                         self.ctx, self.n, self.anc, self.scale, self.dtype)
