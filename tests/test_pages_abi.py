"""CPU checks of free, trim, fork and compact: refusals before anything is
enqueued, workspaces, and the plain definitions that the GPU tests compare
with."""
import ctypes as C

import numpy as np
import pytest

import draft_tree_construction_markov_amd as pct
from pagesref import Pages, check
from test_cache_abi import HEADS, ODD, PAGES, shape

FIELDS = ("ctx_len", "block_table", "n_held", "ring", "ring_state", "extra")
WS = C.c_void_p(1 << 24)


def state(**kw):
    a = {x: 4096 * (i + 1) for i, x in enumerate(FIELDS)}
    a.update(kw)
    return pct._PageState(*a.values())


def ref(x):
    return None if x is None else C.byref(x)


def free(sh, m=3, places=256, st=state(), ws=WS, nbytes=1 << 20):
    return pct.lib().pct_cache_free(ref(sh), m, places, ref(st), ws, nbytes,
                                    None)


def trim(sh, n=None, st=state(), ws=WS, nbytes=1 << 20):
    return pct.lib().pct_cache_trim(ref(sh), n, ref(st), ws, nbytes, None)


def fork(sh, layers=2, stride=10 * 2 * 16 * 64, m=3, st=state(), ws=WS,
         nbytes=1 << 20, **kw):
    a = dict(src=256, dst=512, length=None)
    b = dict(kc=C.c_void_p(256), vc=C.c_void_p(256), done=768)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    return pct.lib().pct_cache_fork(ref(sh), layers, stride, m, *a.values(),
                                    ref(st), *b.values(), ws, nbytes, None)


def compact(sh, layers=2, stride=10 * 2 * 16 * 64, st=state(), out=1 << 20,
            kc=C.c_void_p(256), vc=C.c_void_p(256), ws=WS, nbytes=1 << 20):
    return pct.lib().pct_cache_compact(ref(sh), layers, stride, ref(st), out,
                                       kc, vc, ws, nbytes, None)


CALLS = [free, trim, fork, compact]


@pytest.mark.parametrize("bad", PAGES)
def test_page_sizes_are_checked(bad):
    L = pct.lib()
    for call in CALLS:
        assert call(shape(**bad)) == 1
    assert L.pct_cache_free_workspace(ref(shape(**bad))) == 0
    assert L.pct_cache_fork_workspace(ref(shape(**bad)), 1) == 0
    assert L.pct_cache_compact_workspace(ref(shape(**bad))) == 0


@pytest.mark.parametrize("bad", HEADS)
def test_heads_are_checked(bad):
    assert fork(shape(**bad), stride=1 << 40) == 1
    assert compact(shape(**bad), stride=1 << 40) == 1


@pytest.mark.parametrize("call", CALLS)
def test_refuses(call):
    assert call(None) == 1
    assert call(shape(), st=None) == 1
    for name in FIELDS:
        assert call(shape(), st=state(**{name: None})) == 1, name
        other = 4096 if name != "ctx_len" else 8192
        assert call(shape(), st=state(**{name: other})) == 1, name
    assert call(shape(batch=65536)) == 2
    assert call(shape(n_pages=(1 << 30) + 1), **(
        dict(stride=1 << 50) if call in (fork, compact) else {})) == 2
    assert call(shape(), ws=None) == 3
    assert call(shape(), nbytes=7) == 3
    assert call(shape(), ws=ODD) == 1


WORKSPACE = {free: lambda L, s: L.pct_cache_free_workspace(s),
             trim: lambda L, s: L.pct_cache_free_workspace(s),
             fork: lambda L, s: L.pct_cache_fork_workspace(s, 3),
             compact: lambda L, s: L.pct_cache_compact_workspace(s)}


@pytest.mark.parametrize("call", CALLS)
def test_a_workspace_that_overlaps_is_refused(call):
    need = WORKSPACE[call](pct.lib(), ref(shape()))
    kw = dict(n=256) if call is trim else {}
    arrays = [4096 * (i + 1) for i in range(6)]
    arrays += {free: [256], trim: [256], fork: [256, 512, 768],
               compact: [1 << 20]}[call]
    for x in arrays:
        # the first address that is aligned and whose last bytes meet x
        for y in (x, ((x - need) // 16 + 1) * 16):
            assert y > 0
            assert call(shape(), ws=C.c_void_p(y), **kw) == 1, (x, y)
    if call is fork:
        assert fork(shape(), length=1024, ws=C.c_void_p(1024)) == 1


def test_free_and_trim_refuse():
    assert free(shape(), m=-1) == 1
    assert free(shape(), m=65536) == 2
    assert free(shape(), places=None) == 1
    assert free(shape(), places=4096) == 1
    assert trim(shape(), n=3 * 4096) == 1
    assert free(shape(), m=0, places=None) == 0


@pytest.mark.parametrize("call", [fork, compact])
def test_caches_are_checked(call):
    for kw in (dict(kc=None), dict(vc=None), dict(kc=ODD), dict(vc=ODD),
               dict(layers=0), dict(layers=1025),
               dict(stride=10 * 2 * 16 * 64 - 8),
               dict(stride=10 * 2 * 16 * 64 + 4)):
        assert call(shape(), **kw) == 1, kw


def test_fork_and_compact_refuse():
    for name in ("src", "dst", "done"):
        assert fork(shape(), **{name: None}) == 1
        assert fork(shape(), **{name: 6 * 4096}) == 1
    assert fork(shape(), length=4096) == 1
    assert fork(shape(), done=260) == 1
    assert fork(shape(), m=-1) == 1
    assert fork(shape(), m=65536) == 2
    assert fork(shape(), m=0, src=None, dst=None, done=None) == 0
    need = pct.lib().pct_cache_fork_workspace(ref(shape()), 3)
    assert fork(shape(), nbytes=need - 1) == 3
    assert pct.lib().pct_cache_fork_workspace(ref(shape()), -1) == 0
    assert compact(shape(), out=None) == 1
    assert compact(shape(), out=2 * 4096 + 4) == 1
    assert compact(shape(), out=4096) == 1


def test_definitions_keep_every_page_once():
    rng = np.random.default_rng(0)
    s = Pages(9, 60, 8, 12, head=17)
    s.k = rng.standard_normal((1, 60, 1, 8, 1))
    for b, n in enumerate((30, 16, 0, 5)):
        s.grow(b, n)
    check(s)
    seen = s.k[0, s.table[0, :4], 0].copy()
    done = s.fork([0, 0, 1, 0, 9, 2, 0], [5, 6, 7, 5, 8, 8, 1])
    assert done.tolist() == [1, 1, 1, 0, 0, 0, 0]
    check(s)
    assert s.held.tolist() == [4, 2, 0, 1, 0, 4, 4, 2, 0]
    assert np.array_equal(s.k[0, s.table[5, :4], 0].reshape(-1)[:30],
                          seen.reshape(-1)[:30])
    s.free([0, 0, -1, 99])
    check(s)
    s.ctx[6] = 3
    s.trim(np.full(9, 5), 0)
    check(s)
    assert s.held.tolist() == [0, 2, 0, 1, 0, 4, 1, 2, 0]
    kept = s.k[0, s.table[5, :4], 0].copy()
    s.compact()
    check(s)
    assert s.table.max() == 60 - s.state[1] - 1
    assert np.array_equal(s.k[0, s.table[5, :4], 0], kept)
