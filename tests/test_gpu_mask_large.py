"""A mask of more words than a grid has threads, on the GPU."""
import numpy as np
import pytest
import torch

import draft_tree_construction_markov_amd as pct
from gpu_util import announce

pytestmark = pytest.mark.gpu


def test_more_words_than_a_grid_has_threads():
    # 34 GB: node i's parent is i / 2 - 1, so that paths are short
    batch, N = 4097, 8192
    words = N // 64
    assert batch * N * words > 1 << 32
    one = torch.arange(N, dtype=torch.int32, device="cuda") // 2 - 1
    n = torch.full((batch,), N, dtype=torch.int32, device="cuda")
    n[7], n[batch - 1] = 0, 5000
    out = torch.full((batch, N, words), -1, dtype=torch.int64, device="cuda")
    announce("mask of", batch, N)
    pct.tree_mask(one.expand(batch, N).contiguous(), n, out=out)
    torch.cuda.synchronize()
    want = np.zeros((N, N), bool)
    for i in range(N):
        want[i] = want[i // 2 - 1] if i > 1 else False
        want[i, i] = True
    want = torch.from_numpy(np.packbits(want, axis=1, bitorder="little").view(
        np.int64)).cuda()
    for b in range(batch - 1):
        if b != 7:
            assert torch.equal(out[b], want), b
    assert not out[7].any() and not out[batch - 1, 5000:].any()
    assert torch.equal(out[batch - 1, :5000], want[:5000])
    del out
    torch.cuda.empty_cache()
