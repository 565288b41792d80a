"""GPU checks of pct_tree_attention where a form of its kernels can go wrong by
itself: contexts longer than the block table."""
import numpy as np
import pytest
import torch

from cacheref import Case
from cachestrict import compare
from gpu_util import announce
from test_gpu_cache_attention import device_args, handle

pytestmark = pytest.mark.gpu


def check(c, *what):
    announce("tree attention", what, tuple(c.q.shape), tuple(c.k.shape))
    h = handle(c)
    q, k, v, table, ctx, n, mask = device_args(c)
    out, lse = h.run(q, k, v, table, ctx, n, mask=mask, scale=c.scale)
    torch.cuda.synchronize()
    compare(c, out, lse)


# ---------------------------------------------------------------------------
# contexts longer than the block table

def cut(c, width):
    c.table = np.ascontiguousarray(c.table[:, :width])
    return c


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,chain", [(0, True), (3, False), (20, False),
                                     (70, True)])
@pytest.mark.parametrize("page,width", [(8, 7), (16, 5), (2, 33), (128, 1)])
def test_contexts_longer_than_the_table(D, N, chain, page, width):
    # the table ends inside a tile, the context goes on past it
    end = page * width
    check(cut(Case(D + N, 3, N, 4, 2, D, page, [end + 44, end, 300],
                   n=[N, N, N // 2], chain=chain), width), "cut")


@pytest.mark.parametrize("width", [7, 12])
def test_contexts_longer_than_the_table_in_tiles_of_128_rows(width):
    check(cut(Case(width, 5, 300, 512, 64, 16, 8, [60, 95, 96, 100, 300]),
              width), "cut")
