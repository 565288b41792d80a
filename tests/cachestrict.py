"""The 64-bit definition of attention over a paged cache once more, row by row
of matrices, for long and large calls, and a comparison that lets nothing
pass: every finite value has to be within its tolerance and every other one
equal."""
from __future__ import annotations

import math

import torch

from cacheref import F32, HALF_STEP

LEAST_FP16 = 2.0 ** -24  # least step of fp16
LIFT = 2.0 ** 7  # fp16 probabilities are kept as 2^7 p


def definition(c, device="cuda"):
    """(out, lse, tol, tol_lse) of a cacheref.Case in float64; unused rows
    are zero.

    Tolerances are those of cacheref.attention, with its term for what lies
    below fp16's least step 2^-24 in its exact form: a probability p (of at
    most 1, for the largest score) is held as 2^7 p, so half a step is 2^-32
    of it, and the values that it meets add up to sum |v|; the result's own
    half step is 2^-25."""
    batch, R, Hq, D = c.q.shape
    n_pages, Hkv, page, _ = c.k.shape
    G = Hq // Hkv
    u = HALF_STEP[c.dtype]
    f64 = dict(dtype=torch.float64, device=device)
    out, tol = torch.zeros(batch, R, Hq, D, **f64), torch.zeros(
        batch, R, Hq, D, **f64)
    lse, tol_l = torch.zeros(batch, R, Hq, **f64), torch.zeros(
        batch, R, Hq, **f64)
    table = torch.from_numpy(c.table).to(device).long()
    kc, vc, qd = (x.to(device) for x in (c.k, c.v, c.q))
    for b in range(batch):
        m = int(c.n[b]) + 1
        if m <= 0:
            continue
        ctx = int(c.ctx[b])
        t = torch.arange(min(ctx + m, c.table.shape[1] * page), device=device)
        t = t[(table[b][t // page] >= 0) & (table[b][t // page] < n_pages)]
        node = t - ctx - 1
        see = (node < 0)[None].repeat(m, 1)
        on = node >= 0
        if c.anc is None:
            see[:, on] = node[on][None] < torch.arange(m, device=device)[:, None]
        elif on.any():
            anc = torch.from_numpy(c.anc[b, :m - 1]).to(device)
            see[1:, on] = anc[:, node[on]]
        at, off = table[b][t // page], t % page
        T = see.sum(1, keepdim=True).double()
        for h in range(Hkv):
            K, V = kc[at, h, off].double(), vc[at, h, off].double()
            fine = torch.where(torch.isfinite(V), V, 0.0)
            odd = torch.nonzero(~torch.isfinite(V).all(1)).reshape(-1)
            for g in range(h * G, (h + 1) * G):
                Q = qd[b, :m, g].double()
                S = (Q @ K.T * c.scale).masked_fill_(~see, -math.inf)
                ds = ((Q.abs() @ K.nan_to_num(0, 0, 0).abs().T)
                      .masked_fill_(~see, 0.0).amax(1, keepdim=True)
                      if len(t) else torch.zeros(m, 1, **f64))
                ds *= abs(c.scale) * (D + 3) * F32
                top = (S.amax(1, keepdim=True) if len(t) else
                       torch.full((m, 1), -math.inf, **f64))
                some = T > 0
                p = S.sub_(torch.where(some, top, 0.0)).exp_()
                total = p.sum(1, keepdim=True)
                p /= torch.where(some, total, 1.0)
                o, A = p @ fine, p @ fine.abs()
                for i in odd.tolist():
                    x = torch.where(torch.isfinite(V[i]), 0.0, V[i])
                    hit = see[:, i, None] & (x != 0)[None]
                    o += torch.where(hit, p[:, i, None] * x[None], 0.0)
                out[b, :m, g] = o
                z = torch.where(some, top + total.log(), -math.inf)[:, 0]
                lse[b, :m, g] = z
                steps = (2 * T + 64) * F32
                tol[b, :m, g] = A * (2 * u + torch.expm1(2 * ds) + steps)
                if c.dtype == torch.float16:
                    tol[b, :m, g] += LEAST_FP16 / 2 * (
                        1 + (see.double() @ fine.abs()) / LIFT)
                tol_l[b, :m, g] = (ds + steps)[:, 0] + z.abs() * 8 * F32
    return out, lse, tol, tol_l


def agree(got, want, tol, what):
    got = got.double()
    fine = torch.isfinite(want)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), what
    assert torch.equal(got[~fine & ~nan], want[~fine & ~nan]), what
    off = (got - want).abs()[fine]
    limit = tol[fine]
    assert torch.isfinite(limit).all(), what
    assert (off <= limit).all(), (
        what, int((off > limit).sum()),
        float((off / limit.clamp(min=1e-300)).max()))


def compare(c, out, lse):
    o, z, tol, tol_l = definition(c, out.device)
    agree(out, o, tol, "out")
    agree(lse, z, tol_l, "lse")
