"""GPU checks of the page plan, the row writes and the commit of accepted
paths against plain definitions (equal in every value), and of a whole round
on a paged cache."""
import math

import numpy as np
import pytest
import torch

import draft_tree_construction_markov_amd as pct
from cacheref import HALF_STEP, pack, plan, random_trees
from gpu_util import announce, dev_i32

pytestmark = pytest.mark.gpu


def same(got, want, what):
    assert np.array_equal(got.cpu().numpy(), want), what


class PlanState:
    def __init__(self, rng, batch, width, P, head=0):
        self.table = np.full((batch, width), -1, np.int32)
        self.held = np.zeros(batch, np.int32)
        self.ring = rng.permutation(P).astype(np.int32)
        self.state = np.array([head, P], np.int32)
        self.dev = [dev_i32(x) for x in (self.table, self.held, self.ring,
                                         self.state)]

    def step(self, h, ctx, n, N, page, depth, given=True):
        t, hd, r, st = self.dev
        o = h.run(dev_i32(ctx), dev_i32(n) if given else None, t, hd, r, st,
                  depth=None if N == 0 else dev_i32(depth))
        torch.cuda.synchronize()
        (self.table, self.held, self.ring, self.state), rows = plan(
            ctx, n, N, page, self.table, self.held, self.ring, self.state,
            depth if N > 0 else None)
        for x, y, what in zip(self.dev, (self.table, self.held, self.ring,
                                         self.state),
                              ("table", "held", "ring", "ring_state")):
            same(x, y, what)
        for x, y, what in zip((o.slot, o.pos, o.missing), rows,
                              ("slot", "pos", "missing")):
            same(x, y, what)


@pytest.mark.parametrize("batch,N,page,width,P,hi", [
    (1, 0, 16, 8, 40, 100), (1, 64, 16, 40, 60, 500), (5, 7, 1, 200, 400, 150),
    (33, 30, 8, 40, 700, 250), (8, 1500, 64, 60, 300, 2000),
    (3, 5, 1024, 3, 6, 2500), (1030, 3, 4, 12, 4000, 40),
    (2100, 0, 16, 4, 1500, 60)])
def test_plan_over_rounds(batch, N, page, width, P, hi):
    rng = np.random.default_rng(batch + N)
    h = pct.CachePlan(batch, N, P, page, width)
    s = PlanState(rng, batch, width, P, head=int(rng.integers(P)))
    ctx = rng.integers(0, hi, batch)
    announce("plan", dict(batch=batch, N=N, page=page, P=P))
    for turn in range(6):
        n = rng.integers(-1, N + 1, batch)
        end = rng.random(batch) < 0.3
        ctx = np.where(end, 0, ctx + rng.integers(0, 9, batch))
        n = np.where(end & (rng.random(batch) < 0.5), -1, n)
        depth = random_trees(rng, min(batch, 4), N, np.full(4, N))[1]
        depth = np.resize(depth, (batch, N)).astype(np.int32)
        s.step(h, ctx, n, N, page, depth)
    # everything given back
    s.step(h, np.zeros(batch, int), np.full(batch, -1), N, page, depth)
    assert s.state[1] == P and sorted(s.ring) == list(range(P))


@pytest.mark.parametrize("batch,N", [(64, 31), (64, 32), (64, 0), (65, 0),
                                     (17, 119), (2, 1023), (1, 2048)])
def test_plan_around_the_bounds_of_one_workgroup(batch, N):
    test_plan_over_rounds(batch, N, 16, 90 + N // 16, 4000, 900)


def test_plan_without_nodes_and_out_of_pages():
    rng = np.random.default_rng(1)
    h = pct.CachePlan(4, 6, 10, 4, 5)
    s = PlanState(rng, 4, 5, 10)
    depth = np.ones((4, 6), np.int32)
    full = np.full(4, 6)
    announce("plan out of pages")
    # 7 + 9 tokens: 2 and 4 pages; then 5 pages do not fit, nor does anything
    s.step(h, np.array([1, 9, 13, 1]), full, 6, 4, depth, given=False)
    assert s.held.tolist() == [2, 4, 0, 0]
    s.step(h, np.array([1, 40, 13, 1]), full, 6, 4, depth, given=False)
    assert s.held.tolist() == [2, 5, 0, 0]  # wider than the table
    s.step(h, np.array([0, 0, 0, 1]), np.array([-1, -1, -1, 6]), 6, 4, depth)


@pytest.mark.parametrize("N,page", [(0, 16), (17, 8), (40, 128)])
@pytest.mark.parametrize("Hkv,D,dtype", [(1, 16, torch.float16),
                                         (3, 80, torch.bfloat16),
                                         (8, 128, torch.bfloat16)])
def test_write(N, page, Hkv, D, dtype):
    rng = np.random.default_rng(N + D)
    batch, P = 5, 120
    R = N + 1
    qkv = torch.from_numpy(rng.standard_normal((batch, R, 2 * Hkv + 2, D)))
    qkv = qkv.to(dtype).cuda()
    k, v = qkv[:, :, 1:1 + Hkv], qkv[:, :, 2 + Hkv:]
    slot = rng.permutation(P * page)[:batch * R].reshape(batch, R)
    slot[rng.random(slot.shape) < 0.2] = -1
    slot[0, 0], slot[-1, -1] = P * page, 2 ** 40
    kc = torch.full((P, Hkv, page, D), 5.0, dtype=dtype, device="cuda")
    vc = torch.full_like(kc, 6.0)
    wk, wv = kc.clone(), vc.clone()
    for b in range(batch):
        for i in range(R):
            x = int(slot[b, i])
            if 0 <= x < P * page:
                wk[x // page, :, x % page] = k[b, i]
                wv[x // page, :, x % page] = v[b, i]
    announce("write", dict(N=N, page=page, Hkv=Hkv, D=D))
    pct.cache_write(k, v, torch.from_numpy(slot).cuda(), kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def commit_inputs(rng, batch, N, B, page, layers, Hkv, D, ctx):
    need = -(-(ctx + N + 1) // page)
    P = int(need.sum()) + 2
    perm = rng.permutation(P)
    table = np.full((batch, int(need.max()) + 1), -1, np.int32)
    at = 0
    for b in range(batch):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    k = torch.from_numpy(rng.standard_normal((layers, P, Hkv, page, D)))
    v = torch.from_numpy(rng.standard_normal((layers, P, Hkv, page, D)))
    tau = np.zeros(batch, np.int32)
    acc = np.full((batch, B), -1, np.int32)
    for b in range(batch):
        m = int(rng.integers(0, min(B, N) + 1))
        acc[b, :m] = np.sort(rng.choice(N, m, replace=False)) if m else []
        tau[b] = m + 1
    return table, k, v, tau, acc


def committed(table, k, v, tau, acc, ctx, n, page):
    k, v = k.clone(), v.clone()
    out = ctx.copy()
    for b in range(len(ctx)):
        if n[b] < 0:
            continue
        out[b] += tau[b]
        for j in range(tau[b] - 1):
            f, t = ctx[b] + 1 + acc[b, j], ctx[b] + 1 + j
            pf, pt = table[b, f // page], table[b, t // page]
            if pf < 0 or pt < 0:
                continue
            for c in (k, v):
                c[:, pt, :, t % page] = c[:, pf, :, f % page].clone()
    return k, v, out


@pytest.mark.parametrize("batch,N,B,page,layers,Hkv,D", [
    (1, 8, 4, 16, 1, 1, 16), (6, 64, 7, 16, 3, 2, 64), (3, 300, 200, 8, 2, 2, 48),
    (5, 40, 16, 1, 4, 3, 128), (2, 16, 16, 128, 32, 8, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(batch, N, B, page, layers, Hkv, D, in_place):
    rng = np.random.default_rng(N + B)
    ctx = rng.integers(0, 150, batch)
    table, k, v, tau, acc = commit_inputs(rng, batch, N, B, page, layers,
                                          Hkv, D, ctx)
    n = np.full(batch, N)
    if batch > 2:
        n[1] = -1  # a padded request
        table[2, -2] = -1  # a page that is gone
    k, v = k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda()
    wk, wv, wc = committed(table, k, v, tau, acc, ctx, n, page)
    dctx = dev_i32(ctx)
    announce("commit", dict(batch=batch, N=N, B=B, page=page, layers=layers))
    got = pct.cache_commit(dev_i32(tau), dev_i32(acc), dctx, dev_i32(n),
                           dev_i32(table), k, v,
                           out=dctx if in_place else None)
    torch.cuda.synchronize()
    same(got, wc, "ctx")
    if not in_place:
        same(dctx, ctx, "ctx before")
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_commit_of_the_whole_chain_and_of_nothing():
    rng = np.random.default_rng(8)
    ctx = np.array([4, 9])
    table, k, v, tau, acc = commit_inputs(rng, 2, 20, 20, 4, 1, 1, 16, ctx)
    k, v = k.half().cuda(), v.half().cuda()
    tau[:] = 21, 1
    acc[0], acc[1] = np.arange(20), -1
    before = k.clone(), v.clone()
    announce("commit chain")
    got = pct.cache_commit(dev_i32(tau), dev_i32(acc), dev_i32(ctx), None,
                           dev_i32(table), k[0], v[0])
    torch.cuda.synchronize()
    assert got.tolist() == [25, 10]
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])


def test_commit_stops_at_a_node_outside_the_tree():
    rng = np.random.default_rng(9)
    ctx = np.array([3, 3])
    table, k, v, tau, acc = commit_inputs(rng, 2, 30, 8, 8, 2, 2, 32, ctx)
    n = np.array([30, 5])
    tau[:] = 7, 7
    acc[0] = [1, 4, 2 ** 30, 9, 10, 11, 12, 13]
    acc[1] = [0, 2, 4, 5, 6, 7, 8, 9]
    k, v = k.half().cuda(), v.half().cuda()
    wk, wv, _ = committed(table, k, v, np.array([3, 4]), acc, ctx, n, 8)
    announce("commit outside")
    got = pct.cache_commit(dev_i32(tau), dev_i32(acc), dev_i32(ctx),
                           dev_i32(n), dev_i32(table), k, v)
    torch.cuda.synchronize()
    assert got.tolist() == [10, 10]
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_rounds_on_a_paged_cache_follow_the_plain_sequence():
    """Rounds of build_tree, plan, write, attention, acceptance and commit:
    after each, every request's cache holds the keys and values of its
    committed tokens, and the root's attention is that of plain attention
    over them."""
    rng = np.random.default_rng(12)
    batch, B, V, N, layers, Hq, Hkv, D, page = 3, 4, 200, 14, 2, 4, 2, 32, 8
    dtype = torch.bfloat16
    cache = pct.PagedCache(batch, N, 60, page, 16, Hq, Hkv, D, layers=layers,
                           dtype=dtype)
    # a token's key and value in a layer, from the token alone
    emb = torch.from_numpy(rng.standard_normal((layers, 2, V, Hkv, D)))
    emb = emb.to(dtype).cuda()
    U = torch.from_numpy(rng.standard_normal((V, 16))).float().cuda()
    W = torch.from_numpy(rng.standard_normal((V, 16))).float().cuda()
    root = torch.from_numpy(rng.integers(0, V, batch)).int().cuda()
    text = [[] for _ in range(batch)]
    for turn in range(5):
        L = torch.from_numpy(rng.standard_normal((batch, B, V))).float().cuda()
        tree = pct.build_tree(L, U, W, root, 3, 4, N, mask=True)
        n = tree.n_nodes.clone()
        if turn == 2:
            n[1] = -1  # the request waits for a round
        announce("round", turn)
        rows = cache.plan(n, tree.depth)
        tok = torch.cat([root[:, None], tree.tok.clamp(min=0)], 1).long()
        q = torch.from_numpy(rng.standard_normal((batch, N + 1, Hq, D)))
        q = q.to(dtype).cuda()
        outs = []
        for layer in range(layers):
            cache.write(layer, emb[layer, 0][tok], emb[layer, 1][tok])
            outs.append(cache.attend(layer, q, mask=tree.mask).clone())
        target = torch.from_numpy(rng.integers(0, V, (batch, N + 1))).int()
        for b in range(batch):  # the target agrees with the first child
            for i in reversed(range(int(tree.n_nodes[b]))):
                target[b, int(tree.parent[b, i]) + 1] = int(tree.tok[b, i])
            if turn % 2:
                target[b, int(rng.integers(0, 4))] = int(rng.integers(0, V))
        tau, an, at = pct.verify_accept(tree.tok, tree.parent, tree.depth,
                                        tree.n_nodes, target.cuda(), B,
                                        mask=tree.mask)
        torch.cuda.synchronize()
        assert not rows.missing.any()
        for b in range(batch):
            if n[b] < 0:
                continue
            text[b].append(int(root[b]))
            # the root's attention over the committed text and itself
            for layer in range(layers):
                kk = emb[layer, 0][text[b]].double()
                vv = emb[layer, 1][text[b]].double()
                for h in range(Hq):
                    z = kk[:, h // 2] @ q[b, 0, h].double() * D ** -0.5
                    p = torch.softmax(z, 0)
                    want = p @ vv[:, h // 2]
                    # two roundings, and fp32 sums of at most 64 terms of
                    # scores below 16: far below a third one
                    tol = 3 * HALF_STEP[dtype] * (p @ vv[:, h // 2].abs())
                    got = outs[layer][b, 0, h].double()
                    assert ((got - want).abs() <= tol).all()
            text[b] += at[b, :int(tau[b]) - 1].tolist()
            root[b] = at[b, int(tau[b]) - 1]
        cache.commit(tau, an)
        torch.cuda.synchronize()
        assert cache.ctx_len.tolist() == [len(x) for x in text]
        for b in range(batch):
            p = np.arange(len(text[b]))
            pages = cache.block_table[b].cpu().numpy()[p // page]
            assert (pages >= 0).all()
            for layer in range(layers):
                for c, kind in ((cache.k, 0), (cache.v, 1)):
                    got = c[layer, pages, :, p % page]
                    assert torch.equal(got, emb[layer, kind][text[b]])
    assert min(len(x) for x in text) > 5 and not math.isnan(
        float(outs[0].float().sum()))


def test_a_write_before_the_first_plan_leaves_the_cache():
    cache = pct.PagedCache(2, 3, 8, 16, 4, 4, 2, 32)
    k = torch.ones(2, 4, 2, 32, dtype=torch.bfloat16, device="cuda")
    announce("write before plan")
    cache.write(0, k, k)
    torch.cuda.synchronize()
    assert not cache.k.any() and not cache.v.any()


def test_requests_without_pages_wait_and_go_on():
    """A cache that is too small for its batch: a request that the free ring
    cannot serve keeps its length and its root until pages are given back.
    Whatever was not written, and every page that is given back, is NaN."""
    rng = np.random.default_rng(31)
    batch, N, page, P, layers, Hq, Hkv, D, V = 3, 3, 4, 8, 2, 2, 1, 32, 60
    dtype = torch.bfloat16
    cache = pct.PagedCache(batch, N, P, page, 6, Hq, Hkv, D, layers=layers,
                           dtype=dtype)
    cache.k.fill_(math.nan), cache.v.fill_(math.nan)
    emb = torch.from_numpy(rng.standard_normal((layers, 2, V, Hkv, D)))
    emb = emb.to(dtype).cuda()
    depth = torch.arange(1, N + 1, device="cuda").int().repeat(batch, 1)
    text = [[] for _ in range(batch)]
    root = rng.integers(0, V, batch)
    waited, went_on = np.zeros(batch, bool), 0
    for turn in range(24):
        n = np.full(batch, N)
        gone = []
        if turn % 4 == 3:  # the longest request ends, its place is free
            b = max(range(batch), key=lambda x: len(text[x]))
            gone = [x for x in cache.block_table[b].tolist() if x >= 0]
            cache.ctx_len[b], n[b], text[b], waited[b] = 0, -1, [], False
        draft = rng.integers(0, V, (batch, N))
        announce("waiting round", turn)
        missing = cache.plan(dev_i32(n), depth).missing.tolist()
        if gone:
            cache.k[:, gone], cache.v[:, gone] = math.nan, math.nan
        tok = torch.from_numpy(np.c_[root, draft]).cuda()
        q = torch.from_numpy(rng.standard_normal((batch, N + 1, Hq, D)))
        q = q.to(dtype).cuda()
        outs = []
        for layer in range(layers):
            cache.write(layer, emb[layer, 0][tok], emb[layer, 1][tok])
            outs.append(cache.attend(layer, q).clone())
        taken = rng.integers(0, N + 1, batch)  # whatever the walk answers
        acc = np.where(np.arange(N) < taken[:, None], np.arange(N), -1)
        cache.commit(dev_i32(taken + 1), dev_i32(acc))
        torch.cuda.synchronize()
        for b in range(batch):
            if n[b] < 0:
                continue
            if missing[b] > 0:
                waited[b] = True
                continue
            went_on += int(waited[b])
            waited[b] = False
            for i in range(N + 1):
                see = text[b] + [root[b]] + draft[b, :i].tolist()
                for layer in range(layers):
                    kk = emb[layer, 0][see].double()[:, 0]
                    vv = emb[layer, 1][see].double()[:, 0]
                    for h in range(Hq):
                        z = kk @ q[b, i, h].double() * D ** -0.5
                        p = torch.softmax(z, 0)
                        # two roundings; fp32 sums of some 20 terms of scores
                        # below 16 are far below a third one
                        tol = 3 * HALF_STEP[dtype] * (p @ vv.abs())
                        got = outs[layer][b, i, h].double()
                        assert ((got - p @ vv).abs() <= tol).all()
            text[b] += [root[b]] + draft[b, :taken[b]].tolist()
            root[b] = rng.integers(0, V)
        assert cache.ctx_len.tolist() == [len(x) for x in text], turn
    assert went_on >= 2


@pytest.mark.parametrize("batch,N,P", [(5, 7, 6), (90, 30, 200),
                                       (1030, 3, 900)])
@pytest.mark.parametrize("given", [False, True])
def test_served_nodes(batch, N, P, given):
    rng = np.random.default_rng(batch)
    h = pct.CachePlan(batch, N, P, 8, 20)
    s = PlanState(rng, batch, 20, P)
    some = 0
    announce("served nodes", (batch, N, P, given))
    for turn in range(3):
        ctx = rng.integers(0, 200, batch)
        n = rng.integers(-1, N + 1, batch) if given else np.full(batch, N)
        s.step(h, ctx, n, N, 8, np.ones((batch, N), np.int32), given=given)
        missing = h.out.missing.cpu().numpy()
        same(h.out.n_served, np.where(missing > 0, -1, n), "n_served")
        some += int((missing > 0).sum())
    assert some > 0


def test_a_round_without_a_plan_attends_and_keeps_nothing():
    cache = pct.PagedCache(2, 3, 8, 16, 4, 4, 2, 32)
    q = torch.ones(2, 4, 4, 32, dtype=torch.bfloat16, device="cuda")
    announce("no plan")
    assert not cache.attend(0, q).any()
    cache.commit(dev_i32([3, 1]), dev_i32([[0, 1, -1], [-1, -1, -1]]))
    torch.cuda.synchronize()
    assert cache.ctx_len.tolist() == [0, 0]


def test_commit_stops_at_a_node_outside_trees_of_equal_size():
    rng = np.random.default_rng(10)
    ctx = np.array([3, 6])
    table, k, v, tau, acc = commit_inputs(rng, 2, 30, 5, 8, 2, 2, 32, ctx)
    tau[:] = 5, 6
    acc[0] = [1, 4, 9, 10, -1]  # of trees of 9 nodes: the first two
    acc[1] = [0, 2, 5, 8, 29]   # all but the last
    k, v = k.half().cuda(), v.half().cuda()
    wk, wv, _ = committed(table, k, v, np.array([3, 5]), acc, ctx,
                          np.array([9, 9]), 8)
    announce("commit outside, equal sizes")
    got = pct.cache_commit(dev_i32(tau), dev_i32(acc), dev_i32(ctx), None,
                           dev_i32(table), k, v, N=9)
    torch.cuda.synchronize()
    assert got.tolist() == [8, 12]
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_replayed_rounds_equal_eager_ones():
    # a round captured once, with the lengths, the pages and the requests that
    # wait for pages changing from replay to replay
    rng = np.random.default_rng(44)
    batch, N, page, P, layers, Hq, Hkv, D, B = 5, 20, 8, 26, 2, 4, 2, 64, 6
    make = lambda: pct.PagedCache(batch, N, P, page, 12, Hq, Hkv, D,  # noqa: E731
                                  layers=layers)
    eager, graph = make(), make()
    dt = torch.bfloat16
    buf = dict(n=dev_i32(np.full(batch, N)),
               depth=dev_i32(np.ones((batch, N))),
               mask=torch.zeros(batch, N, 1, dtype=torch.int64, device="cuda"),
               kv=torch.zeros(layers, 2, batch, N + 1, Hkv, D, dtype=dt,
                              device="cuda"),
               q=torch.zeros(batch, N + 1, Hq, D, dtype=dt, device="cuda"),
               tau=dev_i32(np.ones(batch)),
               acc=dev_i32(np.full((batch, B), -1)))

    def one_round(cache):
        rows = cache.plan(buf["n"], buf["depth"])
        out = torch.empty(layers, batch, N + 1, Hq, D, dtype=dt,
                          device="cuda").zero_()
        for layer in range(layers):
            cache.write(layer, *buf["kv"][layer])
            cache.attend(layer, buf["q"], mask=buf["mask"], out=out[layer])
        cache.commit(buf["tau"], buf["acc"])
        return rows, out

    announce("captured rounds")
    with torch.cuda.stream(torch.cuda.Stream()):
        one_round(make())  # what is loaded at the first call
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rows2, out2 = one_round(graph)
    waits = 0
    for turn in range(12):
        n = rng.integers(0, N + 1, batch)
        if turn % 3 == 2:  # a place is emptied
            b = int(rng.integers(batch))
            n[b] = -1
            for cache in (eager, graph):
                cache.ctx_len[b] = 0
        _, depth, anc = random_trees(rng, batch, N, n)
        taken = [int(rng.integers(0, min(B, max(x, 0)) + 1)) for x in n]
        acc = np.full((batch, B), -1, np.int32)
        for b, m in enumerate(taken):
            if m:
                acc[b, :m] = np.sort(rng.choice(n[b], m, replace=False))
        for name, x in (("n", dev_i32(n)), ("depth", dev_i32(depth)),
                        ("mask", torch.from_numpy(pack(anc))),
                        ("kv", torch.from_numpy(rng.standard_normal(
                            tuple(buf["kv"].shape)))),
                        ("q", torch.from_numpy(rng.standard_normal(
                            tuple(buf["q"].shape)))),
                        ("tau", dev_i32(np.array(taken) + 1)),
                        ("acc", dev_i32(acc))):
            buf[name].copy_(x)
        rows, out = one_round(eager)
        g.replay()
        torch.cuda.synchronize()
        waits += int((rows.missing > 0).sum())
        for x, y in ((rows.slot, rows2.slot), (rows.pos, rows2.pos),
                     (rows.missing, rows2.missing),
                     (rows.n_served, rows2.n_served), (out, out2),
                     (eager.ctx_len, graph.ctx_len),
                     (eager.block_table, graph.block_table),
                     (eager.ring, graph.ring), (eager.k, graph.k),
                     (eager.ring_state, graph.ring_state),
                     (eager.v, graph.v)):
            assert torch.equal(x, y), turn
        assert torch.isfinite(out.float()).all()
    assert waits > 0 and int(eager.ctx_len.max()) > 8


def test_the_next_round_may_be_given_the_last_one_s_nodes():
    cache = pct.PagedCache(3, 2, 2, 4, 4, 4, 2, 32)
    n = dev_i32([2, 2, 1])
    depth = dev_i32([[1, 2]] * 3)
    announce("same nodes")
    assert cache.plan(n, depth).missing.tolist() == [0, 0, 1]
    assert cache.n_nodes is n and cache.n_served.tolist() == [2, 2, -1]
    rows = cache.plan(cache.n_nodes, depth)
    torch.cuda.synchronize()
    assert rows.missing.tolist() == [0, 0, 1] and n.tolist() == [2, 2, 1]
    assert cache.n_served.tolist() == [2, 2, -1]
