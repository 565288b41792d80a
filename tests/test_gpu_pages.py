"""GPU checks of free, trim, fork and compact against plain definitions, equal
in every value."""
import dataclasses

import numpy as np
import pytest
import torch

import draft_tree_construction_markov_amd as pct
from gpu_util import announce, dev_i32
from pagesref import Pages, check

pytestmark = pytest.mark.gpu


class Both:
    """The same state here (numpy) and on the GPU."""

    def __init__(self, rng, batch, P, page, width, Hkv=1, D=16, layers=1,
                 dtype=torch.bfloat16, N=0):
        self.s = Pages(batch, P, page, width, head=int(rng.integers(P)))
        self.s.ring = np.roll(rng.permutation(P), 3).astype(np.int32)
        shape = (layers, P, Hkv, page, D)
        self.s.k, self.s.v = (rng.integers(-2 ** 15, 2 ** 15, shape).astype(
            np.int16) for _ in range(2))
        self.k, self.v = (torch.from_numpy(x.copy()).cuda().view(dtype)
                          for x in (self.s.k, self.s.v))
        self.h = pct.CachePages(batch, P, page, width, Hkv, D, layers=layers,
                                dtype=dtype, N=N)

    def up(self):
        s = self.s
        self.d = pct.PageState(*(dev_i32(x) for x in (
            s.ctx, s.table, s.held, s.ring, s.state, s.extra)))

    def same(self):
        torch.cuda.synchronize()
        s = self.s
        for name, want in (("ctx_len", s.ctx), ("n_held", s.held),
                           ("block_table", s.table), ("extra", s.extra),
                           ("ring_state", s.state), ("ring", s.ring)):
            got = getattr(self.d, name).cpu().numpy()
            assert np.array_equal(got, want), name
        for got, want in ((self.k, s.k), (self.v, s.v)):
            assert np.array_equal(got.view(torch.int16).cpu().numpy(), want)

    def free(self, places):
        announce("free", len(places))
        self.s.free(places)
        self.h.free(self.d, dev_i32(places))
        self.same()

    def trim(self, n):
        announce("trim")
        N = self.h.shape.N
        self.s.trim(np.full(self.s.batch, N) if n is None else n, N)
        self.h.trim(self.d, None if n is None else dev_i32(n))
        self.same()

    def fork(self, src, dst, length=None):
        announce("fork", len(src))
        want = self.s.fork(src, dst, length)
        got = self.h.fork(self.d, dev_i32(src), dev_i32(dst), self.k, self.v,
                          length=None if length is None else dev_i32(length))
        self.same()
        assert np.array_equal(got.cpu().numpy(), want)
        return want

    def compact(self, out=False):
        announce("compact")
        to = torch.full_like(self.d.block_table, -9) if out else None
        was = self.d.block_table.clone()
        got = self.h.compact(self.d, self.k, self.v, out=to)
        if out:
            assert got is to and torch.equal(was, self.d.block_table)
            self.d = dataclasses.replace(self.d, block_table=to)
        self.s.compact()
        self.same()


SHAPES = [
    # batch pages page width Hkv D layers ctx
    (4, 40, 16, 6, 2, 64, 3, 60),
    (9, 300, 8, 40, 1, 16, 1, 200),
    (20, 700, 1, 60, 2, 16, 2, 55),
    (70, 2000, 4, 60, 1, 32, 1, 180),      # more places than one workgroup's
    (12, 50, 128, 5, 3, 80, 2, 500),
    (5, 12, 1024, 3, 1, 128, 2, 2500),
    (10, 33000, 2, 900, 1, 16, 1, 1700),   # more pages than one workgroup's
    (1100, 3500, 4, 6, 1, 16, 1, 20),      # more pairs than a workgroup
    (4500, 9000, 4, 4, 1, 16, 1, 12),      # more places than LDS holds
]


@pytest.mark.parametrize("batch,P,page,width,Hkv,D,layers,hi", SHAPES)
def test_over_rounds(batch, P, page, width, Hkv, D, layers, hi):
    rng = np.random.default_rng(batch + P)
    t = Both(rng, batch, P, page, width, Hkv, D, layers,
             dtype=torch.float16 if batch % 2 else torch.bfloat16)
    s = t.s
    for b in range(batch):
        if rng.random() < 0.6 and s.state[1] > P // 3:
            s.grow(b, int(rng.integers(0, hi)))
    t.up()
    for turn in range(4):
        m = max(1, batch // 2)
        src = rng.integers(-1, batch + 1, m)
        dst = rng.integers(-1, batch + 1, m)
        t.fork(src, dst, rng.integers(-3, hi, m) if turn % 2 else None)
        check(s)
        t.free(rng.integers(-2, batch + 2, max(1, batch // 3)))
        check(s)
        # contexts that nobody shares shrink or go on
        for b in range(batch):
            if s.held[b] and not s.extra[s.table[b, :s.held[b]]].any() and \
                    rng.random() < 0.5:
                s.ctx[b] = rng.integers(0, s.ctx[b] + 1)
        t.d.ctx_len.copy_(dev_i32(s.ctx))
        t.trim(rng.integers(-1, 3, batch))
        check(s)
        t.compact(out=turn % 2 == 1)
        check(s)
    t.free(np.arange(batch))
    check(s)
    assert s.state[1] == P


def test_one_source_many_places():
    rng = np.random.default_rng(1)
    t = Both(rng, 130, 400, 16, 40, Hkv=2, D=32)
    t.s.grow(3, 16 * 30 + 5)
    t.up()
    dst = np.array([b for b in range(130) if b != 3])
    assert t.fork(np.full(129, 3), dst).all()
    assert t.s.extra.max() == 129
    t.free(np.arange(129))
    t.free([129, 129])
    check(t.s)
    assert t.s.state[1] == 400


def test_the_ring_runs_out():
    rng = np.random.default_rng(2)
    t = Both(rng, 12, 20, 4, 8)
    t.s.grow(0, 10)
    t.s.grow(1, 8)      # whole pages: needs none of its own
    for b in (2, 3):
        t.s.grow(b, 24)
    t.up()
    assert t.s.state[1] == 3
    done = t.fork([0, 1, 0, 0, 0, 1, 0], [4, 5, 6, 7, 8, 9, 10])
    assert done.tolist() == [1, 1, 1, 1, 0, 1, 0]
    check(t.s)


def test_pairs_that_are_left_out():
    rng = np.random.default_rng(3)
    t = Both(rng, 8, 60, 8, 6)
    t.s.grow(0, 20)
    t.s.grow(1, 9)
    t.s.ctx[2] = 30          # a context whose pages it does not hold
    t.up()
    done = t.fork([0, 0, 0, 2, 7, 0, 1, 5], [0, 1, 4, 5, 6, 4, 3, 7],
                  [20, 20, 0, 30, 30, 8, 900, 5])
    # an empty source makes an empty place
    assert done.tolist() == [0, 0, 1, 0, 1, 0, 1, 1]
    assert t.s.ctx.tolist() == [20, 9, 30, 9, 0, 0, 0, 0]


def test_bad_table_entries():
    rng = np.random.default_rng(4)
    t = Both(rng, 4, 40, 8, 8)
    for b in range(2):
        t.s.grow(b, 37)
    t.s.table[0, 1], t.s.table[0, 2] = -5, 40
    t.s.table[1, 4] = 1 << 30   # the page in part: cannot be copied
    t.up()
    assert t.fork([0, 1], [2, 3]).tolist() == [1, 0]
    t.compact()
    t.free([0, 2])


def test_nothing_to_do():
    rng = np.random.default_rng(5)
    t = Both(rng, 3, 10, 4, 3)
    t.up()
    none = np.zeros(0, np.int32)
    t.free(none)
    t.fork(none, none)
    t.trim(np.full(3, -1))
    t.compact()
    t.free([-1, 3])
    for b in range(3):
        t.s.grow(b, 12 if b < 2 else 8)
    t.s.grow(2, 12)
    t.up()
    t.compact()              # nine of ten pages
    t.compact(out=True)      # once more: nothing moves


def test_trim_keeps_the_pages_of_the_nodes():
    rng = np.random.default_rng(8)
    t = Both(rng, 5, 60, 4, 11, N=9)
    for b, n in enumerate((40, 13, 0, 22)):
        t.s.grow(b, n)
    t.s.ctx[:] = 3, 13, 0, 10, 0
    t.up()
    t.trim(np.array([9, -1, 4, 30, -3]))
    assert t.s.held.tolist() == [4, 4, 0, 5, 0]
    t.s.ctx[:] = 0
    t.up()
    t.trim(None)
    assert t.s.held.tolist() == [3, 3, 0, 3, 0]


def test_graph_and_other_stream():
    rng = np.random.default_rng(6)
    t = Both(rng, 9, 80, 8, 8, Hkv=2, D=32, layers=2)
    for b in range(3):
        t.s.grow(b, 20 + 9 * b)
    t.up()
    src, dst = dev_i32([0, 1, 2, 0]), dev_i32([5, 6, 7, 8])
    done = torch.zeros(4, dtype=torch.int32, device="cuda")

    def step():
        t.h.free(t.d, dst)
        t.h.fork(t.d, src, dst, t.k, t.v, out=done)
        t.h.compact(t.d, t.k, t.v)

    def plain():
        t.s.free([5, 6, 7, 8])
        assert t.s.fork([0, 1, 2, 0], [5, 6, 7, 8]).all()
        t.s.compact()

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    announce("pages, other stream")
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    plain()
    t.same()
    announce("pages, graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        plain()
        t.same()
        assert done.all()
        t.free([0])
        t.s.grow(0, 33)
        for name, x in (("ctx_len", t.s.ctx), ("block_table", t.s.table),
                        ("n_held", t.s.held), ("ring_state", t.s.state)):
            getattr(t.d, name).copy_(dev_i32(x))


def test_binding_refuses():
    rng = np.random.default_rng(7)
    t = Both(rng, 4, 10, 4, 3)
    t.up()
    with pytest.raises(ValueError):
        t.h.free(t.d, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        t.h.fork(t.d, dev_i32([0]), dev_i32([1, 2]), t.k, t.v)
    with pytest.raises(ValueError):
        t.h.fork(t.d, dev_i32([0]), dev_i32([1]), t.k[:, :5], t.v)
    with pytest.raises(ValueError):
        t.h.compact(t.d, t.k, t.v, out=t.d.block_table[:2])
    with pytest.raises(pct.PCTError):      # more pairs than places
        t.h.fork(t.d, dev_i32([0] * 9), dev_i32([1] * 9), t.k, t.v)
    bad = dataclasses.replace(t.d, extra=t.d.ring)
    with pytest.raises(pct.PCTError):
        t.h.trim(bad)
    for kw in (dict(extra=t.d.extra.long()), dict(ring=t.d.ring[:5]),
               dict(n_held=t.d.n_held.cpu()), dict(ctx_len=t.d.ctx_len[:3])):
        with pytest.raises(ValueError):
            dataclasses.replace(t.d, **kw)
    with pytest.raises(ValueError):
        pct.CachePages(4, 10, 4, 2, 1, 16).trim(t.d)
    with pytest.raises(pct.PCTError):
        pct.CachePages(0, 10, 4, 3, 1, 16)


def test_fork_of_many_layers_and_heads():
    # more (layer, head) runs than a grid has rows of workgroups
    rng = np.random.default_rng(9)
    P, layers, Hkv = 4, 1024, 1024
    h = pct.CachePages(3, P, 2, 2, Hkv, 16, layers=layers)
    s = Pages(3, P, 2, 2)
    s.grow(0, 3)
    d = pct.PageState(*(dev_i32(x) for x in (s.ctx, s.table, s.held, s.ring,
                                             s.state, s.extra)))
    k = torch.randint(-99, 99, (layers, P, Hkv, 2, 16),
                      dtype=torch.int16, device="cuda").view(torch.bfloat16)
    v = k.flip(0).contiguous()
    want = [x.view(torch.int16).clone() for x in (k, v)]
    announce("fork, many layers and heads")
    assert h.fork(d, dev_i32([0]), dev_i32([2]), k, v).tolist() == [1]
    assert s.fork([0], [2]).tolist() == [1]
    assert np.array_equal(d.block_table.cpu().numpy(), s.table)
    a, b = int(s.table[0, 1]), int(s.table[2, 1])
    for x, got in zip(want, (k, v)):
        x[:, b, :, :1] = x[:, a, :, :1]
        assert torch.equal(got.view(torch.int16), x)
