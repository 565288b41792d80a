"""GPU checks of the share plan (equal in every value) and of shared attention
against the 64-bit definition of tree attention."""
import math

import numpy as np
import pytest
import torch

import draft_tree_construction_markov_amd as pct
from cacheref import pack
from gpu_util import announce, dev_i32
from shareref import SharedCase, share
from test_gpu_cache_attention import compare
from test_share_abi import two_depths

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


# ---------------------------------------------------------------------------
# plan

def check_plan(ctx, n, table, P, page, N, least, given=True):
    h = pct.SharePlan(len(ctx), N, P, page, table.shape[1], least=least)
    announce("share plan", len(ctx), table.shape, P, page, least)
    o = h.run(dev_i32(ctx), dev_i32(n) if given else None, dev_i32(table))
    torch.cuda.synchronize()
    leader, shared = share(ctx, np.clip(n, -1, N), table, P, page, least)
    assert np.array_equal(o.leader.cpu().numpy(), leader)
    assert np.array_equal(o.shared.cpu().numpy(), shared)
    # the packed rows: each row of a group's requests once, group by group
    batch, R = len(ctx), N + 1
    plan = o.plan.cpu().numpy()
    rows = plan[10 * batch + 4:]
    groups = plan[4 * batch:8 * batch].reshape(batch, 4)
    at, seen = 0, 0
    for g, lead in enumerate(x for x in range(batch)
                             if leader[x] == x and shared[x] > 0):
        want = [b * R + i for b in range(batch) if leader[b] == lead and
                shared[b] > 0 for i in range(int(min(n[b], N)) + 1)]
        assert groups[g].tolist() == [lead, shared[lead], len(want), at]
        assert rows[at:at + len(want)].tolist() == want
        at, seen = at + len(want), g + 1
    assert not groups[seen:, 2].any()
    return leader, shared


def forked_tables(rng, batch, width, page, P, prompts, depth):
    """Tables along random chains of forks, some entries of them replaced."""
    table = np.full((batch, width), -1, np.int32)
    ctx = np.zeros(batch, np.int64)
    for b in range(batch):
        m = int(rng.integers(1, width + 1))
        table[b, :m] = rng.integers(0, P, m)
        ctx[b] = rng.integers((m - 1) * page, m * page)
        if b and rng.random() < 0.8:
            a = int(rng.integers(max(0, b - prompts), b))
            k = min(int(rng.integers(0, depth + 1)), m)
            table[b, :k] = table[a, :k]
    return table, ctx


@pytest.mark.parametrize("batch,width,page,P,prompts,depth,N", [
    (1, 5, 16, 40, 1, 5, 0), (2, 6, 16, 40, 1, 6, 0), (7, 9, 1, 30, 2, 9, 3),
    (33, 40, 8, 3000, 4, 38, 0), (64, 500, 16, 9000, 3, 400, 20),
    (128, 300, 16, 20000, 3, 290, 2), (130, 40, 1024, 500, 9, 40, 0),
    (1024, 20, 4, 5000, 40, 18, 1), (1000, 70, 2, 20000, 6, 60, 20),
    (12, 3000, 16, 30000, 2, 2900, 5), (70, 30, 8, 20, 5, 28, 1),
    (16, 300, 16, 5000, 3, 290, 2), (8, 2000, 16, 9000, 2, 1900, 0)])
def test_plan(batch, width, page, P, prompts, depth, N):
    rng = np.random.default_rng(batch + width)
    groups = 0
    for turn in range(3):
        table, ctx = forked_tables(rng, batch, width, page, P, prompts, depth)
        n = rng.integers(-1, N + 2, batch)
        if turn == 2:
            bad = rng.random(table.shape) < 0.1
            table = np.where(bad, rng.choice([-9, P, 1 << 30], table.shape),
                             table).astype(np.int32)
            ctx = ctx + rng.integers(0, 3 * page, batch)
        shared = check_plan(ctx, n, table, P, page, N,
                            int(rng.integers(1, 20 * page)), given=True)[1]
        groups += int((shared > 0).any())
    assert groups or batch < 10
    check_plan(ctx, np.full(batch, N), table, P, page, N, 1, given=False)


def test_plan_of_equal_and_of_strange_tables():
    table = np.tile(np.arange(12, dtype=np.int32), (40, 1))
    check_plan(np.full(40, 12 * 8), np.zeros(40, int), table, 12, 8, 0, 1)
    # a page at two places, once per request; a page twice in one table
    table = np.array([[0, 1, 2, 3], [1, 0, 2, 3], [0, 1, 2, 3], [5, 5, 5, 5],
                      [5, 5, 5, 5], [2, 1, 0, 3]], np.int32)
    _, shared = check_plan(np.full(6, 16), np.zeros(6, int), table, 6, 4, 0, 1)
    assert shared[0] == shared[2] > 0 and shared[3] == shared[4] > 0
    # lengths past the table, and below zero
    check_plan(np.array([1 << 30, 1 << 30, -5, 2 ** 31 - 1, 16, 15]),
               np.zeros(6, int), table, 6, 4, 0, 1)


# ---------------------------------------------------------------------------
# attention

def run(c, least=1, scale=None, lse=True, q=None, n=None):
    """(out, lse, share) as numpy and the plan's result."""
    batch, R, Hq, D = c.q.shape
    Hkv, width = c.k.shape[1], c.table.shape[1]
    args = (batch, c.N, c.n_pages, c.page, width)
    plan = pct.SharePlan(*args, least=least)
    h = pct.SharedAttention(batch, c.N, Hq, Hkv, D, c.n_pages, c.page, width,
                            dtype=c.dtype, lse=lse)
    mask = None if c.anc is None else torch.from_numpy(pack(c.anc)).cuda()
    table = dev_i32(c.table)
    announce("shared attention", c.q.shape, Hkv, c.page, c.ctx.tolist()[:8])
    h.ws.fill_(0xff)    # NaN wherever it is not written
    s = plan.run(dev_i32(c.ctx), dev_i32(c.n), table)
    out, l = h.run((c.q if q is None else q).cuda(), c.k.cuda(), c.v.cuda(),
                   table, s, mask=mask, scale=c.scale)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), l.double().cpu().numpy(), s


def check(c, got, want=None):
    compare(c, torch.from_numpy(got[0]), torch.from_numpy(got[1]), want)


CASES = [
    # of prefix own N Hq Hkv D page type
    ([0, 0], [40], [3, 9], 0, 4, 4, 64, 16, BF),
    ([0, 0, 0], [64], [1, 64, 30], 0, 8, 2, 128, 16, BF),
    ([0, 1, 0, 1, -1], [100, 333], [5, 17, 40, 0, 60], 0, 8, 1, 128, 16, HF),
    ([0] * 9, [300], [7] * 9, 0, 8, 2, 96, 64, HF),
    ([0] * 20, [130], list(range(20)), 0, 16, 2, 64, 8, BF),
    ([0, 0, 0, 0], [200], [3, 0, 90, 15], 5, 14, 2, 64, 64, HF),
    ([0, 0, 1, 1, -1, -1], [90, 128], [3, 7, 50, 2, 66, 130], 9, 4, 2, 80, 16,
     BF),
    ([0, 0, 0], [257], [10, 70, 128], 33, 4, 1, 128, 32, BF),
    ([0, 0], [150], [20, 3], 64, 4, 2, 128, 16, HF),
    ([0, 0, 0], [129], [1, 2, 3], 20, 2, 1, 192, 16, BF),
    ([0, 0, 0], [129], [1, 2, 3], 40, 4, 1, 256, 16, HF),
    ([0, 0, 0], [100], [4, 5, 6], 3, 3, 3, 256, 16, BF),
    ([0, 0, 0, 0], [61], [4, 5, 6, 9], 6, 4, 2, 48, 4, BF),
    ([0, 0, 0], [77], [4, 5, 6], 30, 4, 2, 64, 2, HF),
    ([0, 0], [5], [1, 1], 2, 2, 2, 16, 1, BF),
    ([-1, -1, -1], [0], [3, 99, 300], 4, 8, 2, 128, 16, BF),
    ([0] * 5, [1100], [1, 1, 1, 1, 1], 0, 4, 4, 64, 1024, BF),
    ([0] * 3, [2100], [1, 400, 9], 1, 2, 1, 64, 16, HF),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in
                                             range(len(CASES))])
@pytest.mark.parametrize("chain", [False, True])
def test_attention(case, chain):
    of, prefix, own, N, Hq, Hkv, D, page, dtype = case
    rng = np.random.default_rng(D + N)
    n = rng.integers(0, N + 1, len(of))
    if len(of) > 3 and chain:
        n[2] = -1
    c = SharedCase(D + N, of, prefix, own, N, Hq, Hkv, D, page, n=n,
                   chain=chain, dtype=dtype)
    got = run(c)
    leader, shared = share(c.ctx, c.n, c.table, c.n_pages, page, 1)
    assert np.array_equal(got[2].shared.cpu().numpy(), shared)
    check(c, got)


def test_many_groups():
    of = [i % 11 if i % 5 else -1 for i in range(60)]
    c = SharedCase(3, of, [16 * (i + 1) for i in range(11)],
                   [i % 40 for i in range(60)], 1, 4, 2, 64, 16)
    got = run(c)
    assert len(set(got[2].leader[got[2].shared > 0].tolist())) == 11
    check(c, got)


@pytest.mark.parametrize("D", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("batch,N,Hq", [(20, 0, 16), (6, 15, 8), (5, 31, 6)])
def test_wide_tables(D, dtype, batch, N, Hq):
    # a block table for long requests: shared row tiles of 128 rows
    of = [i % 2 if i < batch - 1 else -1 for i in range(batch)]
    n = [N - i % (N // 2 + 1) for i in range(batch)]
    c = SharedCase(D + batch, of, [130, 210], [3 + 17 * i % 90 for i in
                                              range(batch)], N, Hq, 2, D, 16,
                   n=n, dtype=dtype)
    wide = np.full((batch, 7000), -1, np.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    got = run(c)
    assert (got[2].shared > 0).sum() == batch - 1
    check(c, got)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
def test_scales(scale):
    c = SharedCase(4, [0, 0, -1, 0], [100], [3, 4, 50, 6], 2, 4, 2, 64, 16,
                   scale=scale)
    check(c, run(c))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_scores_far_apart(dtype):
    # the shared keys dominate some rows, the own keys others
    c = SharedCase(5, [0, 0, 0], [300], [200, 3, 64], 2, 4, 2, 64, 16,
                   dtype=dtype, spread=6.0)
    check(c, run(c))


@pytest.mark.parametrize("N", [0, 5, 40])
def test_missing_pages(N):
    # holes that all requests have, in the shared pages, and others
    c = SharedCase(6, [0, 0, 0], [200], [70, 3, 64], N, 4, 2, 64, 16)
    c.table[:, 3] = -1
    c.table[0, 14], c.table[2, 1:] = c.n_pages, -1
    c.table[2, :3] = c.table[0, :3]
    c.table[2, 4:12] = c.table[0, 4:12]
    got = run(c)
    assert (got[2].shared > 0).all()
    check(c, got)
    # nothing at all
    c.table[:] = -1
    got = run(c)
    assert not got[0].any() and (got[1][:, 0] == -math.inf).all()


def test_what_is_not_finite():
    # in a shared value: reaches all rows of the group, and nobody else
    c = SharedCase(7, [0, 0, -1], [100], [30, 5, 60], 4, 4, 2, 64, 16)
    p, o = int(c.table[0, 2]), 5
    c.v[p, 0, o, 3], c.v[p, 1, o, 7] = math.inf, math.nan
    got = run(c)
    with np.errstate(invalid="ignore"):
        want = c.want()
    check(c, got, want)
    assert np.isposinf(got[0][0, 0, 0, 3]) and np.isnan(got[0][1, 4, 2, 7])
    # in a node's value: its descendants only
    c = SharedCase(8, [0, 0], [64], [30, 5], 6, 4, 2, 64, 16)
    at = int(c.ctx[1]) + 1 + 2
    c.v[int(c.table[1, at // 16]), 0, at % 16, 9] = math.inf
    got = run(c)
    sees = np.concatenate([[False], c.anc[1][:, 2]])
    assert (np.isinf(got[0][1, :, 0, 9]) == sees).all()
    assert np.isfinite(got[0][0]).all()


def test_long_prefix_and_tree_attention_agree():
    c = SharedCase(9, [0] * 8 + [1] * 5 + [-1], [5000, 3500],
                   [1 + 40 * i for i in range(14)], 0, 8, 2, 128, 16)
    got = run(c)
    want = c.want()
    check(c, got, want)
    # and with the other requests' rows there or not, to the bit
    for b in range(1, 8):
        c.n[b] = -1
    alone = run(c)
    check(c, alone, want)


def test_strided_queries_and_out():
    c = SharedCase(10, [0, 0, 0], [100], [3, 40, 60], 3, 4, 2, 64, 16)
    joint = torch.randn(3, 4, 8, 64).to(BF)
    joint[:, :, 2:6] = c.q
    want = run(c)
    got = run(c, q=joint.cuda()[:, :, 2:6])
    assert np.array_equal(want[0], got[0])


def test_runs_repeat_to_the_bit():
    c = SharedCase(11, [0] * 30, [2000], [5 * i for i in range(30)], 0, 8, 2,
                   128, 16)
    x, y = run(c), run(c)
    assert np.array_equal(x[0], y[0]) and np.array_equal(x[1], y[1])


def test_graph_and_other_stream():
    c = SharedCase(12, [0, 0, 0, 1, 1, -1], [300, 100],
                   [20, 3, 64, 9, 11, 80], 2, 4, 2, 64, 16)
    width = c.table.shape[1]
    plan = pct.SharePlan(6, 2, c.n_pages, 16, width, least=1)
    h = pct.SharedAttention(6, 2, 4, 2, 64, c.n_pages, 16, width, lse=True)
    mask = torch.from_numpy(pack(c.anc)).cuda()
    q, k, v, table = c.q.cuda(), c.k.cuda(), c.v.cuda(), dev_i32(c.table)
    ctx, n = dev_i32(c.ctx), dev_i32(c.n)

    def step():
        return h.run(q, k, v, table, plan.run(ctx, n, table), mask=mask)

    def now():
        torch.cuda.synchronize()
        return (h.out.double().cpu().numpy(), h.lse.double().cpu().numpy())

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    announce("shared attention, other stream")
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    check(c, now())
    announce("shared attention, graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for ctx_new, table_new in (
            (c.ctx, c.table), (c.ctx - np.array([0, 0, 200, 0, 20, 0]),
                               c.table),
            (c.ctx, c.table[[0, 0, 2, 3, 4, 5]])):
        c.ctx, c.table = ctx_new, table_new
        c.n = (c.n + 1) % 3
        ctx.copy_(dev_i32(c.ctx))
        n.copy_(dev_i32(c.n))
        table.copy_(dev_i32(c.table))
        c.k.nan_to_num_(0.0)
        c.v.nan_to_num_(0.0)
        k.copy_(c.k)
        v.copy_(c.v)
        h.out.zero_()
        h.lse.zero_()
        g.replay()
        check(c, now())


def test_before_the_first_plan_nothing_is_written():
    plan = pct.SharePlan(3, 2, 10, 16, 4)
    h = pct.SharedAttention(3, 2, 4, 2, 64, 10, 16, 4)
    cache = torch.ones(10, 2, 16, 64, dtype=BF, device="cuda")
    announce("shared attention, no plan")
    out, _ = h.run(torch.ones(3, 3, 4, 64, dtype=BF, device="cuda"), cache,
                   cache, torch.zeros(3, 4, dtype=torch.int32, device="cuda"),
                   plan.out)
    torch.cuda.synchronize()
    assert not out.any()


def test_binding_refuses():
    c = SharedCase(13, [0, 0], [40], [3, 4], 0, 2, 2, 64, 16)
    width = c.table.shape[1]
    h = pct.SharedAttention(2, 0, 2, 2, 64, c.n_pages, 16, width)
    plan = pct.SharePlan(2, 0, c.n_pages, 16, width)
    other = pct.SharePlan(2, 1, c.n_pages, 16, width)
    q, k, v, table = c.q.cuda(), c.k.cuda(), c.v.cuda(), dev_i32(c.table)
    for args in ((q, k, v, table, other.out), (q.cpu(), k, v, table, plan.out),
                 (q, k[:1], v, table, plan.out), (q, k, v.half(), table,
                                                  plan.out),
                 (q, k, v, table[:, :1], plan.out)):
        with pytest.raises(ValueError):
            h.run(*args)
    with pytest.raises(ValueError):
        plan.run(dev_i32([1, 2, 3]), None, table)
    for bad in (dict(batch=1025), dict(batch=0), dict(page_size=3)):
        d = dict(batch=2, N=0, n_pages=4, page_size=16, max_pages=2)
        d.update(bad)
        with pytest.raises(pct.PCTError):
            pct.SharePlan(**d)
        with pytest.raises(pct.PCTError):
            pct.SharedAttention(Hq=2, Hkv=2, D=64, **d)


def test_more_rows_than_a_grid_has():
    # one key-value head for 128 query heads, and as many rows as there are
    N, Hq, page = 8192, 128, 16
    R = N + 1
    table = np.tile(np.arange(514, dtype=np.int32), (2, 1))
    table[1, 1:] += 513
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(1030, 1, page, 16, generator=g, device="cuda").to(BF)
            for _ in range(2))
    q = torch.randn(2, R, Hq, 16, generator=g, device="cuda").to(BF)
    ctx, n, tab = dev_i32([16, 21]), dev_i32([N, 700]), dev_i32(table)
    plan = pct.SharePlan(2, N, 1030, page, 514, least=1)
    h = pct.SharedAttention(2, N, Hq, 1, 16, 1030, page, 514, lse=True)
    announce("shared attention, many rows")
    s = plan.run(ctx, n, tab)
    got, lse = h.run(q, k, v, tab, s)
    assert s.shared.tolist() == [16, 16] and s.leader.tolist() == [0, 0]
    # rows here and there against the definition in 64 bits
    kd, vd = k.double(), v.double()
    for b, i in ((0, 0), (0, 1), (0, 4095), (0, 8192), (0, 8191), (1, 700),
                 (1, 13)):
        t = torch.arange(int(ctx[b]) + i + 1, device="cuda")
        at, off = tab[b].long()[t // page], t % page
        K, V = kd[at, 0, off], vd[at, 0, off]
        z = q[b, i].double() @ K.T * 0.25
        w = torch.softmax(z, -1)
        o, A = w @ V, w @ V.abs()
        ds = (q[b, i].double().abs() @ K.abs().T).max() * 0.25 * 19 * 2 ** -24
        tol = A * (2 * 2 ** -8 + 2 * ds + (2 * len(t) + 64) * 2 ** -24)
        assert ((got[b, i].double() - o).abs() <= tol).all(), (b, i)
        assert ((lse[b, i].double() - torch.logsumexp(z, -1)).abs() <=
                ds + (2 * len(t) + 128) * 2 ** -24).all()
    assert not got[1, 701:].any()


@pytest.mark.parametrize("least", [1, 250 * 8, 250 * 8 + 1])
def test_a_pick_is_measured_by_its_gain(least):
    # (once in one workgroup, once in four launches)
    for wide in (46, 700):
        table = np.full((26, wide), -1, np.int32)
        table[:, :46] = two_depths()
        _, shared = check_plan(np.full(26, 45 * 8), np.zeros(26, int), table,
                               2000, 8, 0, least)
        assert (shared > 0).sum() == (24 if least > 250 * 8 else 26)


SIZES = [
    # of, prefix, own, N, Hq, Hkv, D, page, dtype, table width (0: as needed)
    ([0, 0, 0], [300], [40, 3, 64], 4, 4, 2, 64, 16, BF, 0),
    ([0] * 8 + [1] * 5 + [-1], [5000, 3500], [1 + 40 * i for i in range(14)],
     0, 8, 2, 128, 16, BF, 0),
    ([0, 0, 1, 1, -1], [700, 64], [9, 300, 1, 70, 500], 64, 8, 2, 128, 32, HF,
     0),
    ([0, 0, -1], [250], [10, 90, 30], 256, 2, 1, 128, 16, BF, 0),
    ([0, 0, 0, -1], [400], [5, 60, 7, 200], 40, 8, 2, 192, 16, BF, 0),
    ([0, 0, 1, 1], [200, 130], [5, 60, 7, 33], 70, 8, 2, 128, 16, BF, 7000),
    ([0, 0, 1, 1], [200, 130], [5, 60, 7, 33], 70, 8, 2, 256, 16, HF, 7000)]


@pytest.mark.parametrize("shares", [True, False])
@pytest.mark.parametrize("size", SIZES)
def test_equals_tree_attention(size, shares):
    of, prefix, own, N, Hq, Hkv, D, page, dtype, wide = size
    batch = len(of)
    n = [N - i % (N // 2 + 1) for i in range(batch)]
    c = SharedCase(D + N, of, prefix, own, N, Hq, Hkv, D, page, n=n,
                   dtype=dtype)
    if wide:
        table = np.full((batch, wide), -1, np.int32)
        table[:, :c.table.shape[1]] = c.table
        c.table = table
    # (a promise that no call makes: nobody shares)
    got = run(c, least=1 if shares else 2 ** 31 - 1)
    assert (got[2].shared > 0).any() == shares
    h = pct.TreeAttention(batch, N, Hq, Hkv, D, c.n_pages, page,
                          c.table.shape[1], dtype=dtype, lse=True)
    announce("tree attention of the same rows")
    out, lse = h.run(
        c.q.cuda(), c.k.cuda(), c.v.cuda(), dev_i32(c.table), dev_i32(c.ctx),
        dev_i32(c.n), scale=c.scale,
        mask=None if c.anc is None else torch.from_numpy(pack(c.anc)).cuda())
    torch.cuda.synchronize()
    want = c.want()
    check(c, got, want)
    # each is within its tolerance of the definition: both are within twice it
    # of each other, and unused rows are as they were in both
    used = np.arange(N + 1)[None] <= c.n[:, None]
    for x, y, tol in ((got[0], out, want[2]), (got[1], lse, want[3])):
        y = y.double().cpu().numpy()
        assert (np.abs(x - y)[used] <= 2 * tol[used]).all()
        assert not x[~used].any() and not y[~used].any()
