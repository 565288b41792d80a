"""Plain definition (numpy) of the share plan, and inputs whose requests share
prefixes."""
from __future__ import annotations

import numpy as np
import torch

from cacheref import Case


def share(ctx, n, table, n_pages, page, least):
    """Returns (leader, shared)."""
    batch, width = table.shape
    full = [0 if n[b] < 0 else
            min(max(int(ctx[b]), 0), width * page - 1) // page
            for b in range(batch)]
    count = {}
    for b in range(batch):
        for j, p in enumerate(table[b, :full[b]].tolist()):
            if 0 <= p < n_pages:
                count[j, p] = count.get((j, p), 0) + 1
    pick = {}
    for b in range(batch):
        best, at = 0, -1
        for j in range(full[b]):
            p = int(table[b, j])
            if 0 <= p < n_pages:
                gain = (j + 1) * (count[j, p] - 1)
                if gain > best:
                    best, at = gain, j
        if at >= 0 and best * page >= least:
            pick[b] = at
    leader, shared = np.arange(batch), np.zeros(batch, np.int64)
    groups = {}
    for b in sorted(pick):
        groups.setdefault((pick[b], int(table[b, pick[b]])), []).append(b)
    for members in groups.values():
        lead = members[0]
        d = pick[lead]
        on = [b for b in members
              if np.array_equal(table[b, :d + 1], table[lead, :d + 1])]
        if len(on) > 1:
            leader[on] = lead
            shared[on] = (d + 1) * page
    return leader.astype(np.int32), shared.astype(np.int32)


class SharedCase(Case):
    """Case whose requests share pages: of[b] is the prompt of request b (-1:
    its own), prefix[prompt] its positions, all of them in its requests'
    contexts."""

    def __init__(self, seed, of, prefix, own, N, Hq, Hkv, D, page, n=None,
                 **kw):
        of, own = np.asarray(of), np.asarray(own)
        pre = np.array([prefix[g] if g >= 0 else 0 for g in of])
        super().__init__(seed, len(of), N, Hq, Hkv, D, page, pre + own, n=n,
                         **kw)
        for g in set(of.tolist()) - {-1}:
            members = np.nonzero(of == g)[0]
            lead = members[0]
            whole = prefix[g] // page
            for b in members[1:]:
                # the rest of the prompt is a copy, as a fork makes it
                t = np.arange(whole * page, prefix[g])
                if len(t):
                    at = [torch.from_numpy(self.table[x][t // page].astype(
                        np.int64)) for x in (b, lead)]
                    for c in (self.k, self.v):
                        c[at[0], :, t % page] = c[at[1], :, t % page]
                self.table[b, :whole] = self.table[lead, :whole]
