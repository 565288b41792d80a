"""GPU checks of pct_tree_attention where a form of its kernels can go wrong by
itself: contexts longer than the block table, many small probabilities, rows that a later call does not use,
values and scores that are not finite in every form of the kernels, long
drafts and large trees."""
import math

import numpy as np
import pytest
import torch

from cacheref import Case
from cachestrict import compare
from gpu_util import announce
from test_gpu_cache_attention import device_args, handle, wide

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


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


# ---------------------------------------------------------------------------
# many small probabilities

@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("N,G", [(0, 4), (3, 4), (17, 1), (70, 2)])
@pytest.mark.parametrize("down", [12.0, 17.4, 20.0])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_many_small_probabilities(dtype, N, G, down, at):
    # One key that takes all rows' weight and has no value; the others lie
    # `down` below it and add up to far more than a step of the result.  64
    # requests share their pages: with 8 heads each, no row tile is cut into
    # runs with references of their own.
    ctx, batch, Hkv, D = 32767, 64, 8, 16
    c = Case(N + G, 1, N, G * Hkv, Hkv, D, 64, [ctx], dtype=dtype,
             scale=1.0)
    q = np.zeros((batch, N + 1, G * Hkv, D))
    q[..., 0] = 1.0
    q[..., 1] = c.rng.uniform(-0.05, 0.05, q.shape[:3])
    c.q = torch.from_numpy(q).to(dtype)
    t = np.arange(ctx + N + 1)
    k = np.zeros((len(t), Hkv, D))
    k[..., 1] = c.rng.uniform(-1, 1, k.shape[:2])
    v = c.rng.uniform(0.5, 1.5, k.shape)
    top = {"first": 0, "middle": ctx // 2, "last": ctx}[at]
    k[top, :, 0], v[top] = down, 0.0
    p, o = torch.from_numpy(c.table[0][t // 64].astype(np.int64)), t % 64
    c.k[p, :, o] = torch.from_numpy(k).to(dtype)
    c.v[p, :, o] = torch.from_numpy(v).to(dtype)
    c.batch = batch
    c.table, c.ctx, c.n = (np.repeat(x, batch, 0) for x in (c.table, c.ctx,
                                                            c.n))
    c.anc = None if c.anc is None else np.repeat(c.anc, batch, 0)
    announce("small probabilities", (N, G), down, at)
    q, k, v, table, ctx, n, mask = device_args(c)
    out, lse = handle(c).run(q, k, v, table, ctx, n, mask=mask, scale=1.0)
    torch.cuda.synchronize()
    some = [0, 41]  # requests that are compared
    c.batch, c.q = len(some), c.q[some]
    compare(c, out[some], lse[some])


# ---------------------------------------------------------------------------
# one handle, call after call

@pytest.mark.parametrize("N,G", [(3, 2), (12, 4), (40, 4)])
def test_rows_that_a_later_call_does_not_use_keep_the_earlier_values(N, G):
    first = Case(1, 2, N, 2 * G, 2, 64, 16, [70, 33])
    then = Case(2, 2, N, 2 * G, 2, 64, 16, [70, 33], n=[N // 3, -1])
    width = first.table.shape[1]
    then.table = np.pad(then.table, ((0, 0), (0, width - then.table.shape[1])),
                        constant_values=-1)
    h = handle(first)
    announce("fewer rows", (N, G))
    q, k, v, table, ctx, n, mask = device_args(first)
    out, lse = h.run(q, k, v, table, ctx, n, mask=mask)
    torch.cuda.synchronize()
    compare(first, out, lse)
    kept = out.clone(), lse.clone()
    # the second case's pages behind the first one's
    q, k2, v2, table2, ctx, n, mask = device_args(then)
    P = first.n_pages
    kv = [x.clone() for x in (k, v)]
    assert then.n_pages <= P
    for x, y in zip(kv, (k2, v2)):
        x[:then.n_pages] = y
    again, lse2 = h.run(q, *kv, table2, ctx, n, mask=mask)
    torch.cuda.synchronize()
    assert again is out and lse2 is lse
    for b in range(2):
        m = int(then.n[b]) + 1
        assert torch.equal(out[b, m:], kept[0][b, m:])
        assert torch.equal(lse[b, m:], kept[1][b, m:])
        out[b, m:], lse[b, m:] = 0, 0
    compare(then, out, lse)


# ---------------------------------------------------------------------------
# values and keys that are not finite, in every form of the kernels

# at most 16 rows of a head; row tiles of 64; of 128
FORMS = [(7, 2, False), (3, 4, False), (15, 1, False), (30, 2, False),
         (75, 4, False), (75, 4, True)]


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("N,G,long_table", FORMS)
def test_nodes_that_are_not_finite_reach_their_descendants_only(
        what, dtype, D, N, G, long_table):
    c = Case(D + N, 2, N, 2 * G, 2, D, 16, [45, 127], n=[N, N - 2],
             dtype=dtype)
    nodes = sorted({N // 2, N - 1})  # the first nodes do not see them
    for b in range(2):
        for i in nodes:
            t = int(c.ctx[b]) + 1 + i
            c.v[c.table[b, t // 16], i % 2, t % 16, 5 + i % 8:19] = what
    reached = c.anc[0][:, nodes].any(-1)
    assert reached.any() and not reached.all()
    check(wide(c) if long_table else c, "values", what)


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("N,G,long_table", FORMS)
def test_keys_that_are_not_finite_reach_their_descendants_only(
        what, D, N, G, long_table):
    c = Case(D + N, 2, N, 2 * G, 2, D, 16, [45, 127], n=[N, N - 2])
    for b in range(2):
        t = int(c.ctx[b]) + 1 + N // 2
        c.k[c.table[b, t // 16], :, t % 16, 3] = what
    # (an infinite key gives scores of either sign: exp(inf - inf) where it
    # is the largest, weight 0 where it is the least)
    check(wide(c) if long_table else c, "keys", what)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("N,G,long_table", FORMS)
@pytest.mark.parametrize("ctx", [40, 4000])  # in one run; over several
def test_scores_of_minus_infinity(D, N, G, long_table, ctx):
    # rows that see such scores only are as rows that see nothing; one key
    # with another score takes all the weight
    c = Case(D + N, 2, N, 2 * G, 2, D, 16, [ctx, ctx])
    c.q[..., 0] = 1.0
    t = np.arange(ctx + N + 1)
    for b in range(2):
        p = torch.from_numpy(c.table[b][t // 16].astype(np.int64))
        c.k[p, :, t % 16, 0] = -math.inf
    key = ctx // 3
    p, o = c.table[1, key // 16], key % 16
    c.k[p, :, o, 0] = 0.5
    h = handle(wide(c) if long_table else c)
    q, k, v, table, n_ctx, n, mask = device_args(c)
    announce("scores of -inf", (D, N, G, long_table, ctx))
    out, lse = h.run(q, k, v, table, n_ctx, n, mask=mask)
    torch.cuda.synchronize()
    assert not out[0].any()
    assert (lse[0] == -math.inf).all()
    want = v[p, :, o].repeat_interleave(G, 0).expand_as(out[1])
    assert torch.equal(out[1], want)
    assert torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("where", [0, 50, 100])
@pytest.mark.parametrize("D", [64, 192])
@pytest.mark.parametrize("N,G,long_table", FORMS)
def test_context_values_that_are_not_finite_reach_every_row(where, D, N, G,
                                                            long_table):
    c = Case(D + N, 1, N, 2 * G, 2, D, 16, [100])
    c.v[c.table[0, where // 16], :, where % 16, 9] = math.inf
    check(wide(c) if long_table else c, "context", where)


@pytest.mark.parametrize("D", [160, 192, 256])
@pytest.mark.parametrize("N", [0, 6, 30, 150])
@pytest.mark.parametrize("page,drop", [(1, 0.3), (4, 0.5), (16, 0.4),
                                       (64, 1.0)])
def test_wide_heads_with_missing_and_small_pages(D, N, page, drop):
    check(Case(page + D, 3, N, 4, 2, D, page, [3, 90, 270], drop=drop),
          "pages")


@pytest.mark.parametrize("page", [1, 2, 4])
@pytest.mark.parametrize("N", [5, 60])
def test_nodes_that_are_not_finite_in_small_pages(N, page):
    c = Case(page, 2, N, 4, 2, 192, page, [45, 127])
    for b in range(2):
        t = int(c.ctx[b]) + 1 + 2
        c.v[c.table[b, t // page], :, t % page, 7:9] = math.nan
    check(c, "small pages")


# ---------------------------------------------------------------------------
# long drafts, pieces of prompts and large trees

@pytest.mark.parametrize("N", [1000, 4096, 8192])
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("ctx", [0, 777])
def test_many_rows(N, chain, ctx):
    check(Case(N, 1, N, 2, 1, 64, 16, [ctx], chain=chain), "many rows")


def test_many_rows_of_several_requests():
    check(Case(7, 3, 2500, 4, 2, 128, 16, [100, 0, 2000],
               n=[2500, -1, 1311], dtype=FP16), "many rows")
