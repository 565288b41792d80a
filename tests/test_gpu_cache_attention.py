"""GPU checks of pct_tree_attention against its 64-bit definition: types,
head layouts, lengths from none to long ones, odd sizes, trees, straight
drafts and single tokens, padded requests, pages that are missing, values
that no row sees, strides, streams and captured graphs."""
import math

import numpy as np
import pytest
import torch

import draft_tree_construction_markov_amd as pct
from cacheref import Case, pack
from gpu_util import announce, dev_i32

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def device_args(c):
    return (c.q.cuda(), c.k.cuda(), c.v.cuda(), dev_i32(c.table),
            dev_i32(c.ctx), dev_i32(c.n),
            None if c.anc is None else torch.from_numpy(pack(c.anc)).cuda())


def handle(c, **kw):
    n_pages, Hkv, page, D = c.k.shape
    return pct.TreeAttention(c.batch, c.N, c.q.shape[2], Hkv, D, n_pages,
                             page, c.table.shape[1], dtype=c.dtype, lse=True,
                             **kw)


def compare(c, out, lse, want=None):
    o, z, tol, tol_l = c.want() if want is None else want
    got = out.double().cpu().numpy()
    got_l = lse.double().cpu().numpy()
    for b in range(c.batch):
        m = int(c.n[b]) + 1
        # unused rows are left as they were (zero in a new handle)
        assert not got[b, m:].any() and not got_l[b, m:].any(), b
        g, w, t = got[b, :m], o[b, :m], tol[b, :m]
        assert np.array_equal(np.isnan(g), np.isnan(w)), b
        fine = ~np.isnan(w)
        bad = np.abs(g - w)[fine] > t[fine]
        assert not bad.any(), (b, int(bad.sum()),
                               float((np.abs(g - w)[fine] / np.maximum(
                                   t[fine], 1e-30)).max()))
        gl, wl = got_l[b, :m], z[b, :m]
        assert np.array_equal(np.isnan(gl), np.isnan(wl)), b
        inf = np.isinf(wl)
        assert np.array_equal(gl[inf], wl[inf])
        ok = ~np.isnan(wl) & ~inf
        assert (np.abs(gl - wl)[ok] <= tol_l[b, :m][ok]).all(), b


def check(c):
    announce("tree attention", dict(
        batch=c.batch, N=c.N, q=tuple(c.q.shape), cache=tuple(c.k.shape),
        ctx=c.ctx.tolist()[:8], n=c.n.tolist()[:8], chain=c.anc is None,
        dtype=str(c.dtype)))
    h = handle(c)
    q, k, v, table, ctx, n, mask = device_args(c)
    out, lse = h.run(q, k, v, table, ctx, n, mask=mask, scale=c.scale)
    torch.cuda.synchronize()
    compare(c, out, lse)


@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 128, 160, 192, 256])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("N", [0, 21])
def test_head_sizes(D, dtype, N):
    check(Case(D + N, 3, N, 8, 2, D, 16, [0, 77, 301], dtype=dtype))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (7, 1), (14, 2), (8, 1),
                                    (16, 1), (20, 1), (36, 2), (64, 2),
                                    (12, 3)])
@pytest.mark.parametrize("N", [0, 3, 10])
def test_head_layouts(Hq, Hkv, N):
    check(Case(Hq + N, 2, N, Hq, Hkv, 64, 16, [130, 63]))


@pytest.mark.parametrize("page", [1, 2, 8, 32, 128, 1024])
@pytest.mark.parametrize("N", [0, 40])
def test_page_sizes(page, N):
    check(Case(page, 3, N, 4, 2, 64, page, [5, 200, 333]))


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 31, 32, 33, 63, 64, 65, 127,
                                 128, 129, 255, 256, 257, 511, 513, 1000])
@pytest.mark.parametrize("N,chain", [(0, True), (6, False), (37, True)])
def test_lengths(ctx, N, chain):
    check(Case(ctx * 3 + N, 1, N, 4, 1, 128, 16, ctx, chain=chain))


@pytest.mark.parametrize("N", [1, 2, 7, 8, 15, 16, 31, 32, 63, 64, 65, 127,
                               128, 129, 200])
def test_tree_sizes(N):
    check(Case(N, 2, N, 8, 2, 128, 16, [70, 0], n=[N, N // 2]))


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_uneven_batch_with_padded_requests(chain, dtype):
    n = [33, -1, 0, 1, 12, -1, 32, 5, 33]
    ctx = [0, 100, 1, 700, 64, 0, 1999, 17, 16]
    check(Case(5, 9, 33, 8, 4, 128, 32, ctx, n=n, chain=chain, dtype=dtype))


@pytest.mark.parametrize("N,batch", [(0, 1), (0, 3), (7, 1), (64, 1)])
def test_long_context(N, batch):
    check(Case(N + batch, batch, N, 8, 2, 128, 16, 20011, chain=N == 7))


def test_many_requests():
    rng = np.random.default_rng(3)
    check(Case(9, 70, 4, 4, 2, 64, 16, rng.integers(0, 400, 70),
               n=rng.integers(-1, 5, 70)))


@pytest.mark.parametrize("N", [0, 30])
@pytest.mark.parametrize("page,drop", [(16, 0.4), (4, 0.7), (64, 1.0)])
def test_missing_pages(N, page, drop):
    # dropped pages are not attended; all of them gone: empty rows
    check(Case(page, 4, N, 4, 2, 64, page, [3, 90, 200, 470], drop=drop))


@pytest.mark.parametrize("spread,scale", [(1.0, 0.0), (30.0, None),
                                          (8.0, -0.3), (200.0, 1.0)])
@pytest.mark.parametrize("N", [0, 19])
def test_flat_and_peaked_scores(spread, scale, N):
    check(Case(11, 2, N, 4, 1, 64, 16, [300, 40], spread=spread, scale=scale))


def test_capacity_smaller_than_the_rows():
    # positions past the block table have no page
    c = Case(4, 2, 20, 4, 2, 64, 8, [50, 30])
    c.table = np.ascontiguousarray(c.table[:, :7])
    check(c)


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_a_node_that_is_not_finite_reaches_its_descendants_only(what):
    c = Case(21, 2, 50, 8, 2, 64, 16, [100, 9])
    bad = 3
    for b in range(2):
        t = int(c.ctx[b]) + 1 + bad
        c.v[c.table[b, t // 16], :, t % 16, 5:9] = what
    want = c.want()
    reached = c.anc[:, :, bad]
    assert reached.any() and not reached.all()
    o = want[0][:, 1:]
    assert np.isfinite(o[~reached]).all()
    h = handle(c)
    q, k, v, table, ctx, n, mask = device_args(c)
    announce("not finite", what)
    out, lse = h.run(q, k, v, table, ctx, n, mask=mask)
    torch.cuda.synchronize()
    got = out[:, 1:].double().cpu().numpy()
    # unreached rows are right; reached ones are not finite where V was not
    assert (np.abs(got - o)[~reached] <= want[2][:, 1:][~reached]).all()
    at = np.zeros(64, bool)
    at[5:9] = True
    assert not np.isfinite(got[reached][:, :, at]).any()
    assert (np.abs(got - o)[reached][:, :, ~at] <=
            want[2][:, 1:][reached][:, :, ~at]).all()


def test_a_key_that_is_not_finite_reaches_its_descendants_only():
    c = Case(22, 1, 40, 4, 2, 64, 16, [60])
    t = 60 + 1 + 2
    c.k[c.table[0, t // 16], :, t % 16, 3] = math.nan
    reached = c.anc[0, :, 2]
    o, z, tol, tol_l = c.want()
    h = handle(c)
    q, k, v, table, ctx, n, mask = device_args(c)
    announce("key not finite")
    out, lse = h.run(q, k, v, table, ctx, n, mask=mask)
    torch.cuda.synchronize()
    got = out[0, 1:].double().cpu().numpy()
    assert (np.abs(got - o[0, 1:])[~reached] <= tol[0, 1:][~reached]).all()
    assert np.isnan(got[reached]).all()
    assert np.isnan(lse[0, 1:].cpu().numpy()[reached]).all()


def test_strided_queries_and_given_output():
    c = Case(31, 3, 9, 6, 2, 80, 16, [40, 0, 99])
    h = handle(c)
    q, k, v, table, ctx, n, mask = device_args(c)
    joint = torch.full((3, 10, 10, 80), math.nan, dtype=c.dtype,
                       device="cuda")
    joint[:, :, 2:8] = q
    out = torch.zeros(3, 10, 6, 80, dtype=c.dtype, device="cuda")
    announce("strided queries")
    got, lse = h.run(joint[:, :, 2:8], k, v, table, ctx, n, mask=mask,
                     out=out)
    torch.cuda.synchronize()
    assert got is out and not h.out.any()
    compare(c, got, lse)


def test_unused_rows_are_left_as_they_were():
    c = Case(33, 3, 12, 4, 2, 64, 16, [20, 5, 70], n=[4, -1, 12])
    h = handle(c)
    h.out.fill_(7.0)
    h.lse.fill_(9.0)
    q, k, v, table, ctx, n, mask = device_args(c)
    announce("unused rows")
    out, lse = h.run(q, k, v, table, ctx, n, mask=mask)
    torch.cuda.synchronize()
    for b in range(3):
        m = int(c.n[b]) + 1
        assert (out[b, m:] == 7.0).all() and (lse[b, m:] == 9.0).all()
        out[b, m:], lse[b, m:] = 0, 0
    compare(c, out, lse)


def test_function_without_normalisers_and_nodes():
    c = Case(35, 2, 5, 4, 2, 64, 16, [33, 8])
    q, k, v, table, ctx, n, mask = device_args(c)
    announce("function")
    out, none = pct.tree_attention(q, k, v, table, ctx, mask=mask)
    want, lse = pct.tree_attention(q, k, v, table, ctx, n, mask=mask,
                                   lse=True)
    torch.cuda.synchronize()
    assert none is None and torch.equal(out, want)
    compare(c, out, lse)


def test_same_call_gives_the_same_bits():
    c = Case(37, 4, 30, 8, 2, 128, 16, [900, 3000, 20, 5000])
    q, k, v, table, ctx, n, mask = device_args(c)
    h = handle(c)
    announce("same bits")
    a = [x.clone() for x in h.run(q, k, v, table, ctx, n, mask=mask)]
    for _ in range(3):
        b = h.run(q, k, v, table, ctx, n, mask=mask)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("N", [0, 24])
def test_replayed_graph_follows_lengths_and_pages(N):
    c1 = Case(41, 3, N, 8, 2, 128, 16, [2000, 50, 7])
    c2 = Case(42, 3, N, 8, 2, 128, 16, [31, 1900, 400])
    width = max(c1.table.shape[1], c2.table.shape[1])
    P = max(c1.n_pages, c2.n_pages)
    for c in (c1, c2):
        t = np.full((3, width), -1, np.int32)
        t[:, :c.table.shape[1]] = c.table
        c.table = t
        pad = (P - c.n_pages, *c.k.shape[1:])
        c.k = torch.cat([c.k, torch.full(pad, math.nan, dtype=c.dtype)])
        c.v = torch.cat([c.v, torch.full(pad, math.nan, dtype=c.dtype)])
    args = [device_args(c) for c in (c1, c2)]
    buf = [None if x is None else x.clone() for x in args[0]]
    h = handle(c1)
    announce("graph", N)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h.run(*buf[:6], mask=buf[6])
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = h.run(*buf[:6], mask=buf[6])
    for turn in (1, 0, 1, 0):
        c = (c1, c2)[turn]
        for x, y in zip(buf, args[turn]):
            if x is not None:
                x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        compare(c, out, lse)


def test_two_handles_on_two_streams():
    cases = [Case(51, 2, 16, 8, 2, 128, 16, [3000, 40]),
             Case(52, 4, 0, 8, 2, 128, 16, [900, 5000, 1, 64])]
    args = [device_args(c) for c in cases]
    hs = [handle(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    announce("two streams")
    for _ in range(4):
        for h, a, s in zip(hs, args, streams):
            with torch.cuda.stream(s):
                h.run(*a[:6], mask=a[6])
    torch.cuda.synchronize()
    for c, h in zip(cases, hs):
        compare(c, h.out, h.lse)


def test_cache_offsets_past_32_bits():
    # 2^31 elements and more in each cache
    page, Hkv, D = 16, 8, 128
    n_pages = (1 << 31) // (page * Hkv * D) + 64
    c = Case(61, 2, 5, 8, Hkv, D, page, [100, 33])
    q, k, v, table, ctx, n, mask = device_args(c)
    big = [torch.empty(n_pages, Hkv, page, D, dtype=c.dtype, device="cuda")
           for _ in range(2)]
    assert big[0].numel() > 1 << 31
    first = n_pages - c.n_pages
    for x, y in zip(big, (k, v)):
        x[first:] = y
    moved = torch.where(table >= 0, table + first, table)
    h = pct.TreeAttention(2, 5, 8, Hkv, D, n_pages, page, table.shape[1],
                          dtype=c.dtype, lse=True)
    announce("large cache", n_pages)
    out, lse = h.run(q, *big, moved, ctx, n, mask=mask)
    torch.cuda.synchronize()
    compare(c, out, lse)


@pytest.mark.parametrize("D", [80, 192, 256])
@pytest.mark.parametrize("N,ctx", [(70, [0, 200]), (150, [63, 5]),
                                   (129, [31, 700])])
def test_large_trees_of_other_heads(D, N, ctx):
    check(Case(D + N, 2, N, 4, 2, D, 16, ctx, n=[N, N - 7]))


@pytest.mark.parametrize("N,G", [(4, 4), (16, 1), (7, 4), (10, 3), (8, 4),
                                 (15, 4), (16, 4)])
@pytest.mark.parametrize("chain", [False, True])
def test_rows_around_the_bounds_of_the_tiles(N, G, chain):
    check(Case(N * G, 3, N, 2 * G, 2, 128, 16, [2001, 31, 700],
               n=[N, N // 2, N], chain=chain))


@pytest.mark.parametrize("batch,N,Hq,Hkv,hi", [
    (3, 90, 8, 2, 900),      # fewer row tiles than runs
    (40, 40, 32, 8, 60),     # more
    (3, 3, 4, 2, 3000)])     # few rows
def test_workspace_may_hold_anything(batch, N, Hq, Hkv, hi):
    # lengths change from call to call, and with them the row tiles that a
    # request has and those that are cut
    rng = np.random.default_rng(batch + N)
    h = None
    for turn in range(3):
        c = Case(71 + turn, batch, N, Hq, Hkv, 64, 16,
                 rng.integers(0, hi, batch),
                 n=rng.integers(-1, N + 1, batch))
        q, k, v, table, ctx, n, mask = device_args(c)
        new = handle(c)
        if h is not None and h.ws.numel() >= new.ws.numel():
            new.ws.copy_(h.ws[:new.ws.numel()])  # what the last call left
        else:
            new.ws.random_(0, 256)
        h = new
        announce("workspace", (batch, N, turn))
        out, lse = h.run(q, k, v, table, ctx, n, mask=mask)
        torch.cuda.synchronize()
        compare(c, out, lse)
        out.zero_(), lse.zero_()
        h.ws.random_(0, 256)
        h.run(q, k, v, table, ctx, n, mask=mask)
        torch.cuda.synchronize()
        compare(c, out, lse)


def test_values_that_are_not_finite_in_large_trees():
    # nodes in several key tiles, shared tiles of 128 rows
    c = Case(81, 1, 180, 8, 2, 128, 16, [45])
    bad = [0, 30, 77, 150]
    for i in bad:
        t = 46 + i
        c.v[c.table[0, t // 16], :, t % 16, 64:70] = math.inf
    want = c.want()
    reached = c.anc[0][:, bad].any(-1)
    assert reached.any() and not reached.all()
    h = handle(c)
    q, k, v, table, ctx, n, mask = device_args(c)
    announce("not finite, large tree")
    out, lse = h.run(q, k, v, table, ctx, n, mask=mask)
    torch.cuda.synchronize()
    got = out[0, 1:].double().cpu().numpy()
    o, tol = want[0][0, 1:], want[2][0, 1:]
    at = np.zeros(128, bool)
    at[64:70] = True
    assert (np.abs(got - o)[~reached] <= tol[~reached]).all()
    assert np.isinf(got[reached][:, :, at]).all()
    assert (np.abs(got - o)[reached][:, :, ~at] <=
            tol[reached][:, :, ~at]).all()


def wide(c):
    """The same case with a block table for long requests, so that the shape
    asks for row tiles of 128 rows whatever the lengths are."""
    width = 64 * 6300 // c.k.shape[2]
    t = np.full((c.batch, width), -1, np.int32)
    t[:, :c.table.shape[1]] = c.table
    c.table = t
    return c


@pytest.mark.parametrize("D", [16, 64, 80, 96, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_wide_tables_head_sizes(D, dtype):
    check(wide(Case(D + 3, 3, 37, 8, 2, D, 16, [0, 77, 301], dtype=dtype)))


@pytest.mark.parametrize("N", [16, 31, 32, 63, 64, 65, 127, 128, 129, 200,
                               256])
@pytest.mark.parametrize("chain", [False, True])
def test_wide_tables_tree_sizes(N, chain):
    check(wide(Case(N + 1, 3, N, 8, 2, 128, 16, [70, 0, 1291],
                    n=[N, N // 2, N - 1], chain=chain)))


@pytest.mark.parametrize("page", [1, 4, 8, 64, 1024])
@pytest.mark.parametrize("drop", [0.0, 0.5])
def test_wide_tables_pages(page, drop):
    check(wide(Case(page + 7, 3, 40, 4, 2, 64, page, [5, 200, 333],
                    drop=drop)))


def test_wide_tables_uneven_batch():
    n = [33, -1, 0, 40, 12, -1, 32, 5, 33]
    ctx = [0, 100, 1, 700, 64, 0, 1999, 17, 16]
    check(wide(Case(6, 9, 40, 8, 4, 128, 32, ctx, n=n)))


@pytest.mark.parametrize("batch", [2, 70])
def test_wide_tables_more_row_tiles_than_runs(batch):
    rng = np.random.default_rng(batch)
    N, Hkv = (300, 128) if batch == 2 else (40, 4)
    check(wide(Case(batch, batch, N, 4 * Hkv, Hkv, 16, 16,
                    rng.integers(0, 90, batch),
                    n=rng.integers(-1, N + 1, batch))))


@pytest.mark.parametrize("spread,scale", [(30.0, None), (8.0, -0.3),
                                          (200.0, 1.0)])
def test_wide_tables_peaked_scores(spread, scale):
    check(wide(Case(12, 2, 39, 4, 1, 128, 16, [700, 40], spread=spread,
                    scale=scale)))


def test_wide_tables_values_that_are_not_finite():
    c = Case(82, 1, 180, 8, 2, 128, 16, [45])
    bad = [0, 30, 77, 150]
    for i in bad:
        t = 46 + i
        c.v[c.table[0, t // 16], :, t % 16, 64:70] = math.inf
    wide(c)
    want = c.want()
    reached = c.anc[0][:, bad].any(-1)
    h = handle(c)
    q, k, v, table, ctx, n, mask = device_args(c)
    announce("not finite, wide table")
    out, lse = h.run(q, k, v, table, ctx, n, mask=mask)
    torch.cuda.synchronize()
    got = out[0, 1:].double().cpu().numpy()
    o, tol = want[0][0, 1:], want[2][0, 1:]
    at = np.zeros(128, bool)
    at[64:70] = True
    assert reached.any() and not reached.all()
    assert (np.abs(got - o)[~reached] <= tol[~reached]).all()
    assert np.isinf(got[reached][:, :, at]).all()
    assert (np.abs(got - o)[reached][:, :, ~at] <=
            tol[reached][:, :, ~at]).all()
