"""Rounds of a shared paged cache on the GPU: requests are forked, freed and
moved together, rows are rotated into the cache, attended and kept, against a
simulation that keeps every request's keys and values apart."""
import numpy as np
import pytest
import torch

import draft_tree_construction_markov_amd as pct
from cacheref import attention, pack, random_trees
from gpu_util import announce, dev_i32
from pagesref import Pages, check
from rotaryref import rotate, tolerance

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
N, HQ, HKV, D, PAGE, LAYERS = 5, 4, 2, 64, 8, 2


class Rounds:
    def __init__(self, batch, n_pages, width, seed):
        self.rng = np.random.default_rng(seed)
        self.batch = batch
        self.c = pct.PagedCache(batch, N, n_pages, PAGE, width, HQ, HKV, D,
                                layers=LAYERS, share=True, least=1)
        self.rotary = pct.Rotary(D, rot=32)
        self.f = [int(x) % (1 << 64) for x in self.rotary.table.tolist()]
        # what each place's positions hold, per layer: [len][HKV][D]
        none = torch.zeros(0, HKV, D, dtype=BF)
        self.k = [[none] * LAYERS for _ in range(batch)]
        self.v = [[none] * LAYERS for _ in range(batch)]

    def lengths(self):
        return self.c.ctx_len.cpu().numpy()

    def pages(self):
        """Every page is free or held, and counted right."""
        c, s = self.c, Pages.__new__(Pages)
        s.P, s.batch = c.ring.numel(), self.batch
        s.table, s.held, s.ring, s.state, s.extra = (
            x.cpu().numpy() for x in (c.block_table, c.n_held, c.ring,
                                      c.ring_state, c.extra))
        check(s)

    def fork(self, pairs, length=None):
        src, dst = (dev_i32([p[i] for p in pairs]) for i in range(2))
        announce("fork", pairs)
        done = self.c.fork(src, dst, None if length is None
                           else dev_i32(length)).cpu().numpy()
        for i, (a, b) in enumerate(pairs):
            if done[i]:
                m = self.lengths()[b]
                for x in (self.k, self.v):
                    x[b] = [y[:m].clone() for y in x[a]]
        self.pages()
        return done

    def free(self, places):
        announce("free", places)
        self.c.free(dev_i32(places))
        for b in places:
            for x in (self.k, self.v):
                x[b] = [y[:0] for y in x[b]]
        assert not self.lengths()[places].any()
        self.pages()

    def compact(self):
        announce("compact")
        self.c.compact()
        self.pages()
        used = self.c.ring.numel() - int(self.c.ring_state[1])
        held = self.c.n_held.cpu().numpy()
        table = self.c.block_table.cpu().numpy()
        assert all(table[b, :held[b]].max(initial=-1) < used
                   for b in range(self.batch))

    def round(self, n):
        """Plan, write, attend and commit; returns the requests served."""
        c, batch, rng = self.c, self.batch, self.rng
        n = np.asarray(n)
        _, depth, anc = random_trees(rng, batch, N, n)
        announce("round", n.tolist(), self.lengths().tolist())
        rows = c.plan(dev_i32(n), dev_i32(depth))
        served = c.n_served.cpu().numpy()
        assert ((served == n) | (served == -1)).all()
        mask = torch.from_numpy(pack(anc)).cuda()
        ctx = self.lengths()
        new = []
        for layer in range(LAYERS):
            qkv = torch.randn(batch, N + 1, HQ + 2 * HKV, D).to(BF).cuda()
            q, k = qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HKV]
            v = qkv[:, :, HQ + HKV:]
            rq = c.write_rotary(layer, self.rotary, q, k, v)
            out = torch.full((batch, N + 1, HQ, D), 9.0, dtype=BF,
                             device="cuda")
            c.attend(layer, rq, mask, out=out)
            torch.cuda.synchronize()
            pos = rows.pos.cpu().numpy()
            y, mag = rotate(k.float().cpu().numpy(), np.maximum(pos, 0),
                            self.f, 32, "half")
            tol = tolerance(y, mag, BF)
            new.append(v.cpu())
            slot = rows.slot.cpu().numpy()
            keys = torch.zeros(batch, N + 1, HKV, D, dtype=BF)
            for b in range(batch):
                for i in range(served[b] + 1):
                    p, o = divmod(int(slot[b, i]), PAGE)
                    keys[b, i] = c.k[layer, p, :, o].cpu()
                    err = np.abs(keys[b, i].float().numpy() - y[b, i])
                    assert (err <= tol[b, i]).all()
            new.append(keys)
            self.check_attention(layer, rq, v.cpu(), keys, out, ctx, served,
                                 anc)
        # the accepted path: some node and its ancestors
        tau = np.zeros(batch, np.int64)
        accept = np.full((batch, N), -1, np.int64)
        for b in range(batch):
            path = []
            if n[b] > 0 and rng.random() < 0.8:
                path = np.nonzero(anc[b, rng.integers(n[b])])[0].tolist()
            tau[b] = len(path) + 1
            accept[b, :len(path)] = path
            if served[b] >= 0:
                keep = [0] + [1 + x for x in path]
                for layer in range(LAYERS):
                    v, k = new[2 * layer], new[2 * layer + 1]
                    self.k[b][layer] = torch.cat([self.k[b][layer],
                                                  k[b, keep]])
                    self.v[b][layer] = torch.cat([self.v[b][layer],
                                                  v[b, keep]])
        c.commit(dev_i32(tau), dev_i32(accept))
        want = np.where(served >= 0, ctx + tau, ctx)
        assert np.array_equal(self.lengths(), want)
        self.pages()
        return served

    def check_attention(self, layer, q, v, k, out, ctx, served, anc):
        """Against the 64-bit definition over caches of one page a request."""
        width = int(max(ctx.max() + N + 1, 1))
        kc = torch.full((self.batch, HKV, width, D), float("nan"),
                        dtype=torch.float64)
        vc = kc.clone()
        for b in range(self.batch):
            m = int(ctx[b])
            for cache, old, rows in ((kc, self.k, k), (vc, self.v, v)):
                cache[b, :, :m] = old[b][layer].double().transpose(0, 1)
                cache[b, :, m:m + served[b] + 1] = \
                    rows[b, :served[b] + 1].double().transpose(0, 1)
        table = np.arange(self.batch)[:, None]
        o, _, tol, _ = attention(q.double().cpu().numpy(), kc.numpy(),
                                 vc.numpy(), table, ctx, served, anc,
                                 D ** -0.5, BF)
        got = out.double().cpu().numpy()
        for b in range(self.batch):
            m = served[b] + 1
            assert (np.abs(got[b, :m] - o[b, :m]) <= tol[b, :m]).all(), b
            assert (got[b, m:] == 9.0).all()


def test_rounds():
    r = Rounds(9, 300, 24, 0)
    x = -1
    for _ in range(4):
        r.round([5, 3, 0, x, x, x, x, x, x])
    # a prompt of many positions, then samples of it
    for _ in range(12):
        r.round([5, 5, x, x, x, x, x, x, x])
    done = r.fork([(0, 3), (0, 4), (0, 5), (1, 6), (0, 3), (7, 8)])
    assert done.tolist() == [1, 1, 1, 1, 0, 1]
    for _ in range(3):
        r.round([5, 4, 3, 2, 1, 0, 5, x, x])
        assert (r.c.share.shared > 0).sum() == 6
    # a step of a search: some end, others take their places
    r.free([3, 5, 7])
    r.fork([(4, 3), (6, 5), (6, 7)], [1000, 20, 13])
    r.compact()
    for _ in range(2):
        r.round([2, x, 2, 2, 2, 2, 2, 2, 1])
    r.free([0])           # the first holder goes, the others stay
    r.round([x, 1, 1, 1, 1, 1, 1, 1, 1])
    r.free(list(range(9)))
    assert int(r.c.ring_state[1]) == 300 and not r.c.extra.any()


def test_a_place_is_emptied_by_its_lengths():
    r = Rounds(3, 60, 10, 1)
    for _ in range(5):
        r.round([5, -1, -1])
    r.fork([(0, 1), (0, 2)])
    r.c.ctx_len[0] = 0
    for x in (r.k, r.v):
        x[0] = [y[:0] for y in x[0]]
    r.round([-1, 3, 3])
    r.round([2, 3, 3])


def test_requests_that_wait_share_nothing():
    r = Rounds(4, 8, 10, 2)
    for _ in range(4):
        r.round([5, -1, -1, -1])
    while r.lengths()[0] < 40:
        r.round([5, -1, -1, -1])
    r.fork([(0, 1), (0, 2)])
    served = r.round([5, 5, 5, 5])
    assert (served == -1).any() and (served >= 0).any()
    r.free([2])
    r.round([0, 0, -1, 0])


def test_nothing_until_the_next_plan():
    r = Rounds(3, 60, 10, 3)
    for _ in range(4):
        r.round([5, 5, -1])
    c = r.c
    for act in (lambda: c.fork(dev_i32([0]), dev_i32([2])),
                lambda: c.free(dev_i32([2])), c.compact):
        c.plan(dev_i32([2, 2, -1]), dev_i32(np.ones((3, N))))
        act()
        before = [x.clone() for x in (c.k, c.v, c.ctx_len)]
        kv = torch.ones(3, N + 1, HKV, D, dtype=BF, device="cuda")
        out = torch.full((3, N + 1, HQ, D), 3.0, dtype=BF, device="cuda")
        c.write(0, kv, kv)
        c.attend(0, torch.ones_like(out), out=out)
        c.commit(dev_i32([2, 2, 2]), dev_i32(np.zeros((3, 4))))
        torch.cuda.synchronize()
        assert (out == 3.0).all()
        for x, y in zip(before, (c.k, c.v, c.ctx_len)):
            assert torch.equal(x, y)


def test_caches_without_shares_refuse():
    c = pct.PagedCache(2, 0, 8, 8, 4, HQ, HKV, D)
    with pytest.raises(ValueError):
        c.fork(dev_i32([0]), dev_i32([1]))
    with pytest.raises(ValueError):
        c.free(dev_i32([0]))
    with pytest.raises(ValueError):
        c.compact()


def test_captured_rounds_equal_eager_ones():
    batch, n_pages, width = 5, 90, 12
    torch.manual_seed(1)
    rng = np.random.default_rng(4)
    eager, graph = (pct.PagedCache(batch, N, n_pages, PAGE, width, HQ, HKV, D,
                                   share=True, least=1) for _ in range(2))
    rotary = pct.Rotary(D)
    n = torch.zeros(batch, dtype=torch.int32, device="cuda")
    depth = torch.zeros(batch, N, dtype=torch.int32, device="cuda")
    mask = torch.zeros(batch, N, 1, dtype=torch.int64, device="cuda")
    qkv = torch.zeros(batch, N + 1, HQ + 2 * HKV, D, dtype=BF, device="cuda")
    q, k, v = qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HKV], qkv[:, :, HQ + HKV:]
    tau = torch.ones(batch, dtype=torch.int32, device="cuda")
    accept = torch.full((batch, N), -1, dtype=torch.int32, device="cuda")
    outs = [torch.zeros(batch, N + 1, HQ, D, dtype=BF, device="cuda")
            for _ in range(2)]
    turned = [torch.zeros_like(x) for x in outs]

    def step(c, i):
        c.plan(n, depth)
        c.write_rotary(0, rotary, q, k, v, out=turned[i])
        c.attend(0, turned[i], mask, out=outs[i])
        c.commit(tau, accept)

    def inputs(nodes):
        _, d, anc = random_trees(rng, batch, N, np.asarray(nodes))
        n.copy_(dev_i32(nodes))
        depth.copy_(dev_i32(d))
        mask.copy_(torch.from_numpy(pack(anc)).cuda())
        qkv.normal_()
        for b in range(batch):
            path = ([] if nodes[b] < 1 else
                    np.nonzero(anc[b, rng.integers(nodes[b])])[0].tolist())
            tau[b] = len(path) + 1
            accept[b] = torch.tensor((path + [-1] * N)[:N])

    inputs([5, 2, -1, -1, -1])
    for i, c in enumerate((eager, graph)):
        step(c, i)
    g = torch.cuda.CUDAGraph()
    announce("captured shared rounds")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    state = [x.clone() for x in (graph.ctx_len, graph.block_table,
                                 graph.n_held, graph.ring, graph.ring_state)]
    with torch.cuda.graph(g):
        step(graph, 1)
    for x, y in zip((graph.ctx_len, graph.block_table, graph.n_held,
                     graph.ring, graph.ring_state), state):
        assert torch.equal(x, y)         # a capture runs nothing
    live = [5, 2, -1, -1, -1]
    for turn in range(14):
        inputs(live)
        step(eager, 0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(*outs) and torch.equal(*turned)
        for x in ("ctx_len", "block_table", "n_held", "ring", "ring_state",
                  "extra", "k", "v"):
            assert torch.equal(getattr(eager, x), getattr(graph, x)), x
        assert torch.equal(eager.share.shared, graph.share.shared)
        if turn == 5:
            for c in (eager, graph):
                assert c.fork(dev_i32([0, 0]), dev_i32([2, 4])).all()
            live = [5, 2, 4, -1, 3]
        if turn == 9:
            for c in (eager, graph):
                c.free(dev_i32([1, 2]))
                c.fork(dev_i32([4]), dev_i32([3]))
                c.compact()
            live = [1, -1, -1, 5, 5]
    assert (eager.share.shared > 0).sum() == 3


def test_two_caches_on_two_streams():
    torch.manual_seed(2)
    caches = [pct.PagedCache(6, 0, 400, 16, 60, 8, 2, D, share=True, least=1)
              for _ in range(2)]
    rotary = pct.Rotary(D)
    rows = [torch.randn(40, 6, 1, 12, D, device="cuda").to(BF)
            for _ in range(2)]
    outs = [[None] * 40, [None] * 40]
    only = dev_i32([0, -1, -1, -1, -1, -1])
    every = dev_i32([0] * 6)

    def run(i, at):
        c = caches[i]
        x = rows[i][at]
        c.plan(only if at < 20 else every)
        r = c.write_rotary(0, rotary, x[:, :, :8], x[:, :, 8:10],
                           x[:, :, 10:])
        outs[i][at] = c.attend(0, r).clone()
        c.commit(dev_i32([1] * 6), dev_i32(np.full((6, 1), -1)))
        if at == 19:
            c.fork(dev_i32([0] * 5), dev_i32([1, 2, 3, 4, 5]))

    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    announce("two shared caches on two streams")
    for at in range(40):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                run(i, at)
    torch.cuda.synchronize()
    both = [[x.clone() for x in y] for y in outs]
    kept = [c.k.clone() for c in caches]
    # the same, one after the other
    caches = [pct.PagedCache(6, 0, 400, 16, 60, 8, 2, D, share=True, least=1)
              for _ in range(2)]
    for i in range(2):
        for at in range(40):
            run(i, at)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs[i], both[i]))
        assert torch.equal(caches[i].k, kept[i])


def test_no_rows_and_no_groups_until_the_next_plan():
    r = Rounds(4, 60, 10, 3)
    while r.lengths()[0] < 2 * PAGE:
        r.round([5, 5, -1, -1])
    assert r.fork([(0, 2)]).tolist() == [1]
    c = r.c
    for act in (lambda: c.fork(dev_i32([1]), dev_i32([3])),
                lambda: c.free(dev_i32([3])), c.compact):
        rows = c.plan(dev_i32([2, 2, 2, -1]), dev_i32(np.ones((4, N))))
        assert (rows.pos[:3, :3] >= 0).all()
        assert c.share.leader.tolist() == [0, 1, 0, 3]
        assert (c.share.shared > 0).tolist() == [True, False, True, False]
        announce("until the next plan")
        act()
        before = [x.clone() for x in (c.k, c.v)]
        kv = torch.ones(4, N + 1, HKV, D, dtype=BF, device="cuda")
        q = torch.ones(4, N + 1, HQ, D, dtype=BF, device="cuda")
        out = torch.full_like(q, 3.0)
        c.write_rotary(0, r.rotary, q, kv, kv, out=out)
        torch.cuda.synchronize()
        assert (out == 3.0).all()
        for x, y in zip(before, (c.k, c.v)):
            assert torch.equal(x, y)
        assert c.share.leader.tolist() == [0, 1, 2, 3]
        assert not c.share.shared.any()
        assert (rows.pos == -1).all() and (rows.slot == -1).all()
    # and the next plan brings them back
    r.round([2, 2, 2, -1])
    assert c.share.leader.tolist() == [0, 1, 0, 3]


def test_captured_forks_frees_and_compactions_equal_eager_ones():
    batch, n_pages, width = 5, 80, 12
    torch.manual_seed(3)
    eager, graph = (pct.PagedCache(batch, 0, n_pages, PAGE, width, HQ, HKV, D,
                                   layers=LAYERS, share=True, least=1)
                    for _ in range(2))
    src, dst, gone = dev_i32([0, 0]), dev_i32([2, 4]), dev_i32([-1, -1])
    n = dev_i32([0, 0, -1, -1, -1])
    names = ("ctx_len", "block_table", "n_held", "ring", "ring_state", "extra",
             "k", "v", "n_served")

    def move(c):
        c.free(gone)
        done = c.fork(src, dst)
        c.compact()
        return done

    def grow(rounds):
        for _ in range(rounds):
            kv = torch.randn(2, batch, 1, HKV, D, device="cuda").to(BF)
            q = torch.randn(batch, 1, HQ, D, device="cuda").to(BF)
            outs = []
            for c in (eager, graph):
                c.plan(n)
                for layer in range(LAYERS):
                    c.write(layer, kv[0], kv[1] * (layer + 1))
                outs.append(c.attend(LAYERS - 1, q))
                c.commit(dev_i32([1] * batch), dev_i32([[-1]] * batch))
            assert torch.equal(*outs)

    def same():
        torch.cuda.synchronize()
        for x in names:
            assert torch.equal(getattr(eager, x), getattr(graph, x)), x
        for x in ("leader", "shared", "plan"):
            assert torch.equal(getattr(eager.share, x), getattr(graph.share, x))
        assert graph.share.leader.tolist() == list(range(batch))
        assert not graph.share.shared.any()

    grow(3 * PAGE + 2)
    announce("captured forks, frees and compactions")
    state = {x: getattr(graph, x).clone() for x in names}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        done = move(graph)
    for x in names:
        assert torch.equal(getattr(graph, x), state[x]), x  # nothing ran
    for live, pairs, free in (
            ([0, 0, 0, -1, 0], ([0, 0], [2, 4]), [-1, 9]),
            ([0, 0, 0, 0, 0], ([2, 2], [3, 4]), [4, 1]),
            ([0, -1, 0, 0, 0], ([1, 3], [0, 1]), [0, 0]),
            ([-1, 0, 0, 0, 0], ([4, 1], [0, 1]), [1, 0])):
        src.copy_(dev_i32(pairs[0]))
        dst.copy_(dev_i32(pairs[1]))
        gone.copy_(dev_i32(free))
        want = move(eager)
        g.replay()
        assert torch.equal(want, done)
        same()
        n.copy_(dev_i32(live))
        grow(PAGE - 1)


def test_a_plan_that_is_refused_changes_nothing():
    r = Rounds(3, 60, 10, 5)
    while r.lengths()[0] < 2 * PAGE:
        r.round([5, 5, -1])
    r.fork([(0, 2)])
    c = r.c
    depth = dev_i32(np.ones((3, N)))
    for n in ([5, 5, 5], [5, 5, -1]):
        given = dev_i32(n)
        rows = c.plan(given, depth)
        names = ("ctx_len", "block_table", "n_held", "ring", "ring_state",
                 "extra", "n_served")
        before = [getattr(c, x).clone() for x in names]
        slot = rows.slot.clone()
        none = dev_i32([-1, -1, -1])
        for bad in ((none, None), (none, depth[:, 1:]), (none, depth.long()),
                    (none, depth.cpu()), (none[:2], depth),
                    (none.long(), depth), (none.cpu(), depth),
                    (c.n_served, depth)):
            announce("refused plan")
            with pytest.raises(pct.PCTError if bad[0] is c.n_served
                               else ValueError):
                c.plan(*bad)
            torch.cuda.synchronize()
            for x, y in zip(before, (getattr(c, x) for x in names)):
                assert torch.equal(x, y)
            assert torch.equal(slot, rows.slot) and c.n_nodes is given
    r.round([5, 4, 3])
