"""CPU checks beside those of the paged-cache calls: the second 64-bit
definition of attention gives what the first one gives, its comparison lets no
wrong value pass, and refusals of arguments."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import cachestrict
import draft_tree_construction_markov_amd as pct
from cacheref import Case


@pytest.mark.parametrize("kw", [{}, dict(chain=True), dict(drop=0.5),
                                dict(dtype=torch.float16), dict(cut=3)])
def test_both_definitions_agree(kw):
    width = kw.pop("cut", None)
    c = Case(3, 3, 12, 4, 2, 16, 8, [9, 0, 33], n=[12, -1, 5], **kw)
    if width:
        c.table = np.ascontiguousarray(c.table[:, :width])
    a = c.want()
    b = [x.numpy() for x in cachestrict.definition(c, "cpu")]
    for q in range(3):
        m = int(c.n[q]) + 1
        assert not b[0][q, m:].any() and not b[1][q, m:].any()
        for x, y in zip(a[:2], b[:2]):
            assert np.allclose(x[q, :m], y[q, :m], rtol=0, atol=1e-12)
        # no tolerance is wider than the first definition's
        for x, y in zip(a[2:], b[2:]):
            seen = np.isfinite(b[1][q, :m])
            assert (y[q, :m][seen] <= x[q, :m][seen] * (1 + 1e-9)).all()


def test_the_definition_with_values_that_are_not_finite():
    c = Case(5, 1, 9, 2, 1, 16, 8, [20])
    t = 20 + 1 + 4
    c.v[c.table[0, t // 8], 0, t % 8, 3:5] = math.inf
    o, z, tol, _ = cachestrict.definition(c, "cpu")
    sees = torch.from_numpy(np.r_[False, c.anc[0][:, 4]])
    assert sees.any() and not sees.all()
    assert torch.isinf(o[0, sees][..., 3:5]).all()
    assert torch.isfinite(o[0, ~sees]).all() and torch.isfinite(tol).all()
    assert torch.isfinite(o[0, sees][..., 5:]).all()
    assert torch.isfinite(z).all()


def test_the_comparison_lets_nothing_pass():
    want = torch.tensor([1.0, math.inf, math.nan, 0.0], dtype=torch.float64)
    tol = torch.tensor([0.1, math.nan, math.nan, 0.0], dtype=torch.float64)
    cachestrict.agree(want.clone(), want, tol, "same")
    for i, x in ((0, 1.2), (0, math.nan), (0, math.inf), (1, -math.inf),
                 (1, 3.0), (1, math.nan), (2, 0.0), (3, 1e-30)):
        got = want.clone()
        got[i] = x
        with pytest.raises(AssertionError):
            cachestrict.agree(got, want, tol, i)
    tol[0] = math.inf  # a tolerance that is none
    with pytest.raises(AssertionError):
        cachestrict.agree(want, want, tol, "tolerance")


def served(n_served, **kw):
    sh = pct.CacheShape(2, 8, 10, 16, 4, 4, 2, 64, pct.PCT_BF16)
    p = dict(ctx=4096, n=8192, depth=256, table=256, held=256, ring=256,
             state=256, slot=256, pos=256, missing=256)
    p.update(kw)
    return pct.lib().pct_cache_plan_served(
        C.byref(sh), *(C.c_void_p(x) for x in p.values()),
        C.c_void_p(n_served), C.c_void_p(256), 16, None)


def test_served_nodes_do_not_overlap_what_is_read():
    # (16 bytes of workspace are too few: a call that passes the checks of
    # its arguments ends there, before anything is enqueued)
    for bad in (4096, 4100, 4092, 8192, 8188, 8196):
        assert served(bad) == 1, bad
    for good in (None, 4096 + 8, 4096 - 8, 8192 + 8, 256):
        assert served(good) == 3, good
    assert served(0x10000, n=None) == 3
    assert served(0x10000, missing=None) == 1


def attend(scale):
    sh = pct.CacheShape(2, 8, 10, 16, 4, 4, 2, 64, pct.PCT_BF16)
    p = C.c_void_p(256)
    return pct.lib().pct_tree_attention(
        C.byref(sh), scale, p, 256, p, p, p, p, None, None, p, None, p, 16,
        None)


def test_scales_whose_product_with_log2_e_is_not_finite():
    # scores are taken to base 2: 3.4e38 / 1.4427 = 2.36e38
    for bad in (2.4e38, -2.4e38, 3.4e38):
        assert attend(bad) == 1, bad
    for good in (2.3e38, -2.3e38, 0.0, 1e-45):
        assert attend(good) == 3, good  # (too little workspace)


def commit(out, ctx=4096, n=8192, tau=0x10000, accept=0x20000, B=4):
    sh = pct.CacheShape(2, 8, 10, 16, 4, 4, 2, 64, pct.PCT_BF16)
    p = C.c_void_p
    return pct.lib().pct_cache_commit(
        C.byref(sh), 1, 0, B, p(tau), p(accept), p(n), p(256), p(ctx),
        p(0x1001), p(256), p(out), None)


def test_new_lengths_do_not_overlap_what_is_read():
    # (the cache's address is odd: a call that passes the overlaps' checks
    # would still be refused, so the messages tell them apart)
    def refused(*a, **kw):
        assert commit(*a, **kw) == 1
        return b"overlaps" in pct.lib().pct_last_error()

    for bad in (8192, 8188, 8196, 0x10000, 0x10004, 0xfffc, 0x20000, 0x2001c,
                0x1fffc, 4092, 4100):
        assert refused(bad), hex(bad)
    for good in (4096, 8184, 8200, 0x10008, 0xfff8, 0x20020, 0x1fff8):
        assert not refused(good), hex(good)
    assert not refused(8192, n=None)
