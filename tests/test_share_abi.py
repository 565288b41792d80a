"""CPU checks of the share plan and shared attention: refusals before anything
is enqueued, sizes, and the plan's plain definition."""
import ctypes as C
import math

import numpy as np
import pytest

import draft_tree_construction_markov_amd as pct
from shareref import share
from test_cache_abi import D, HEADS, ODD, PAGES, shape

WS = C.c_void_p(1 << 24)


def two_depths():
    """Tables of 46 entries of 26 requests: 10 common pages, and 40 of the
    last 24."""
    table = 50 + np.arange(26 * 46, dtype=np.int32).reshape(26, 46)
    table[:, :10] = np.arange(10)
    table[2:, 10:40] = np.arange(10, 40)
    return table


def plan(sh, least=64, ws=WS, nbytes=1 << 20, **kw):
    a = dict(ctx=256, n=None, table=4096, leader=8192, shared=12288,
             share=C.c_void_p(1 << 20))
    a.update(kw)
    return pct.lib().pct_cache_share(None if sh is None else C.byref(sh),
                                     least, *a.values(), ws, nbytes, None)


def attend(sh, scale=1.0, qs=256, ws=D, nbytes=1 << 40, **kw):
    a = dict(q=D, kc=D, vc=D, table=D, share=D, mask=None, out=D, lse=None)
    a.update(kw)
    return pct.lib().pct_shared_attention(
        None if sh is None else C.byref(sh), scale, a["q"], qs, a["kc"],
        a["vc"], a["table"], a["share"], a["mask"], a["out"], a["lse"], ws,
        nbytes, None)


@pytest.mark.parametrize("bad", PAGES)
def test_page_sizes_are_checked(bad):
    L, sh = pct.lib(), C.byref(shape(**bad))
    assert plan(shape(**bad)) == 1 and attend(shape(**bad)) == 1
    assert L.pct_cache_share_size(sh) == 0
    assert L.pct_cache_share_workspace(sh) == 0
    assert L.pct_shared_attention_workspace(sh) == 0


@pytest.mark.parametrize("bad", HEADS + [dict(Hq=5), dict(Hq=2048, Hkv=2)])
def test_heads_are_checked(bad):
    assert attend(shape(**bad), qs=1 << 20) == 1
    assert pct.lib().pct_shared_attention_workspace(
        C.byref(shape(**bad))) == 0


def test_what_is_too_large_is_unsupported():
    for big in (shape(batch=1025), shape(batch=65536)):
        assert plan(big) == 2 and attend(big) == 2
        assert pct.lib().pct_cache_share_size(C.byref(big)) == 0
    # packed rows in 32 bits
    wide = shape(batch=1024, N=8192, Hq=1024, Hkv=4, D=16)
    assert attend(wide, qs=1 << 20) == 2
    assert pct.lib().pct_shared_attention_workspace(C.byref(wide)) == 0
    assert pct.lib().pct_shared_attention_workspace(
        C.byref(shape(batch=1024))) > 0


def test_plan_refuses():
    assert plan(None) == 1
    for name in ("ctx", "table", "leader", "shared", "share"):
        assert plan(shape(), **{name: None}) == 1, name
    assert plan(shape(), least=0) == 1
    assert plan(shape(), share=ODD) == 1
    for kw in (dict(leader=260), dict(shared=4100), dict(leader=12292),
               dict(n=8192), dict(shared=252)):
        assert plan(shape(), **kw) == 1, kw
    need = pct.lib().pct_cache_share_workspace(C.byref(shape()))
    assert plan(shape(), nbytes=need - 1) == 3
    assert plan(shape(), ws=None) == 3
    assert plan(shape(), ws=ODD) == 1


def test_a_pick_is_measured_by_its_gain():
    """26 requests share 10 pages, 24 of them 40: these pick the deeper page,
    and the other two, whose gain counts all 26, are a group that saves 10
    pages."""
    table = two_depths()
    n, ctx = [0] * 26, [45 * 8] * 26
    for least in (1, 250 * 8):
        leader, shared = share(ctx, n, table, 2000, 8, least)
        assert leader.tolist() == [0, 0] + [2] * 24
        assert shared.tolist() == [80, 80] + [320] * 24
    leader, shared = share(ctx, n, table, 2000, 8, 250 * 8 + 1)
    assert leader.tolist() == [0, 1] + [2] * 24
    assert shared.tolist() == [0, 0] + [320] * 24


def test_plan_refuses_a_share_or_workspace_that_overlaps():
    L, sh = pct.lib(), shape()
    size = L.pct_cache_share_size(C.byref(sh))
    need = L.pct_cache_share_workspace(C.byref(sh))
    # (the first address that is aligned and whose last bytes meet the array)
    at = dict(ctx=256, n=512, table=4096, leader=8192, shared=12288)
    for x in at.values():
        for y in (x, ((x - size) // 16 + 1) * 16):
            assert plan(sh, n=512, share=C.c_void_p(y)) == 1, (x, y)
        for y in (x, ((x - need) // 16 + 1) * 16):
            assert plan(sh, n=512, ws=C.c_void_p(y)) == 1, (x, y)
    assert plan(sh, n=512, share=C.c_void_p(4096 + 16)) == 1   # within
    for y in (WS.value, WS.value + (need - 1) // 16 * 16,
              WS.value - (size - 1) // 16 * 16):
        assert plan(sh, share=C.c_void_p(y)) == 1, y


def test_attention_refuses():
    assert attend(None) == 1
    for name in ("q", "kc", "vc", "table", "share", "out"):
        assert attend(shape(), **{name: None}) == 1, name
    for name in ("q", "kc", "vc", "share", "out"):
        assert attend(shape(), **{name: ODD}) == 1, name
    for qs in (248, 260):
        assert attend(shape(), qs=qs) == 1
    for scale in (math.inf, math.nan, 3e38):
        assert attend(shape(), scale=scale) == 1
    need = pct.lib().pct_shared_attention_workspace(C.byref(shape()))
    assert attend(shape(), nbytes=need - 1) == 3
    assert attend(shape(), ws=None) == 3
    assert attend(shape(), ws=ODD) == 1


def test_definition_by_hand():
    x = -1
    table = np.array([
        [1, 2, 3, 4, x],      # a prompt of 3 pages
        [1, 2, 3, 5, x],
        [1, 2, 6, 7, x],      # shares two pages of it
        [8, 9, 10, 11, 12],   # another prompt of 4
        [8, 9, 10, 11, 13],
        [14, 15, x, x, x],
        [1, 2, 3, 16, x]])    # waits
    n = [0, 0, 0, 0, 0, 0, -1]
    ctx = [16, 17, 18, 19, 19, 5, 16]
    leader, shared = share(ctx, n, table, 17, 4, 4)
    # requests 0 and 1: 2 pages with one more or 3 with each other (gains 4
    # and 3): all three take the two pages
    assert leader.tolist() == [0, 0, 0, 3, 3, 5, 6]
    assert shared.tolist() == [8, 8, 8, 16, 16, 0, 0]
    n[6] = 0
    leader, shared = share(ctx, n, table, 17, 4, 4)
    # three requests by three pages (gain 6) as well as four by two: the first
    assert leader.tolist() == [0, 0, 0, 3, 3, 5, 0]
    assert shared.tolist() == [8, 8, 8, 16, 16, 0, 8]
    # what a group must save
    assert share(ctx, n, table, 17, 4, 25)[1].tolist() == [0] * 7
    assert share(ctx, n, table, 17, 4, 24)[1].tolist() == [8, 8, 8, 0, 0, 0, 8]
    # the root's page is not shared, whole pages of the context are
    assert share([8, 8], [0, 0], np.array([[1, 2, 3], [1, 2, 3]]), 4, 4, 1
                 )[1].tolist() == [8, 8]
    assert share([12, 40], [0, 0], np.array([[1, 2, 3], [1, 2, 3]]), 4, 4, 1
                 )[1].tolist() == [8, 8]
