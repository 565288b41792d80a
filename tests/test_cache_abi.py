"""CPU checks of the paged-cache calls: bad arguments are refused on the host
before anything is enqueued, sizes of workspaces, and the binding's own
checks; pins of the 64-bit definitions that the GPU tests compare with."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import cacheref
import draft_tree_construction_markov_amd as pct

D = C.c_void_p(256)
ODD = C.c_void_p(264)


def shape(**kw):
    d = dict(batch=2, N=8, n_pages=10, page_size=16, max_pages=4, Hq=4, Hkv=2,
             D=64, dtype=pct.PCT_BF16)
    d.update(kw)
    return pct.CacheShape(**d)


PAGES = [dict(batch=0), dict(N=-1), dict(N=8193), dict(n_pages=0),
         dict(page_size=0), dict(page_size=24), dict(page_size=2048),
         dict(max_pages=0), dict(max_pages=1 << 27)]
HEADS = [dict(Hkv=0), dict(Hkv=2048, Hq=2048), dict(D=8), dict(D=72),
         dict(D=272), dict(dtype=0), dict(dtype=7)]


def plan(sh, ws=D, nbytes=1 << 20, **kw):
    a = dict(ctx=D, n=None, depth=D, table=D, held=D, ring=D, state=D, slot=D,
             pos=D, missing=D)
    a.update(kw)
    return pct.lib().pct_cache_plan(None if sh is None else C.byref(sh),
                                    *a.values(), ws, nbytes, None)


def write(sh, ks=128, vs=128, **kw):
    a = dict(k=D, v=D, slot=D, kc=D, vc=D)
    a.update(kw)
    return pct.lib().pct_cache_write(
        None if sh is None else C.byref(sh), a["k"], ks, a["v"], vs,
        a["slot"], a["kc"], a["vc"], None)


def attend(sh, scale=1.0, qs=256, ws=D, nbytes=1 << 40, **kw):
    a = dict(q=D, kc=D, vc=D, table=D, ctx=D, n=None, mask=None, out=D,
             lse=None)
    a.update(kw)
    return pct.lib().pct_tree_attention(
        None if sh is None else C.byref(sh), scale, a["q"], qs, a["kc"],
        a["vc"], a["table"], a["ctx"], a["n"], a["mask"], a["out"], a["lse"],
        ws, nbytes, None)


def commit(sh, layers=2, stride=10 * 2 * 16 * 64, B=4, **kw):
    a = dict(tau=D, acc=D, n=None, table=D, ctx=D, kc=D, vc=D,
             out=C.c_void_p(4096))
    a.update(kw)
    return pct.lib().pct_cache_commit(
        None if sh is None else C.byref(sh), layers, stride, B, *a.values(),
        None)


@pytest.mark.parametrize("bad", PAGES)
def test_page_sizes_are_checked(bad):
    assert plan(shape(**bad)) == 1
    assert attend(shape(**bad)) == 1
    assert commit(shape(**bad)) == 1
    if "max_pages" not in bad:
        assert write(shape(**bad)) == 1
    assert pct.lib().pct_last_error()
    assert pct.lib().pct_tree_attention_workspace(
        C.byref(shape(**bad))) == 0


@pytest.mark.parametrize("bad", HEADS)
def test_heads_are_checked(bad):
    assert write(shape(**bad), ks=1 << 20, vs=1 << 20) == 1
    assert attend(shape(**bad), qs=1 << 20) == 1
    assert commit(shape(**bad), stride=1 << 40) == 1
    assert pct.lib().pct_tree_attention_workspace(
        C.byref(shape(**bad))) == 0


def test_large_batches_are_unsupported():
    big = shape(batch=65536)
    assert plan(big) == 2 and write(big) == 2
    assert attend(big) == 2 and commit(big) == 2
    assert pct.lib().pct_cache_plan_workspace(65536) == 0
    assert pct.lib().pct_cache_plan_workspace(0) == 0


def test_plan_refuses():
    assert plan(None) == 1
    for name in ("ctx", "table", "held", "ring", "state", "slot", "missing",
                 "depth"):
        assert plan(shape(), **{name: None}) == 1, name
    need = pct.lib().pct_cache_plan_workspace(2)
    assert need > 0
    assert plan(shape(), nbytes=need - 1) == 3
    assert plan(shape(), ws=None) == 3
    assert plan(shape(), ws=ODD) == 1


def test_write_refuses():
    assert write(None) == 1
    for name in ("k", "v", "slot", "kc", "vc"):
        assert write(shape(), **{name: None}) == 1, name
    for name in ("k", "v", "kc", "vc"):
        assert write(shape(), **{name: ODD}) == 1, name
    for ks, vs in ((120, 128), (128, 120), (132, 128), (128, 132)):
        assert write(shape(), ks=ks, vs=vs) == 1


def test_attention_refuses():
    assert attend(None) == 1
    for name in ("q", "kc", "vc", "table", "ctx", "out"):
        assert attend(shape(), **{name: None}) == 1, name
    for name in ("q", "kc", "vc", "out"):
        assert attend(shape(), **{name: ODD}) == 1, name
    assert attend(shape(Hq=5), qs=320) == 1
    assert attend(shape(Hq=2048, Hkv=2), qs=1 << 20) == 1
    for qs in (248, 260):
        assert attend(shape(), qs=qs) == 1
    for scale in (math.inf, -math.inf, math.nan):
        assert attend(shape(), scale=scale) == 1
    need = pct.lib().pct_tree_attention_workspace(C.byref(shape()))
    assert need > 0
    assert attend(shape(), nbytes=need - 1) == 3
    assert attend(shape(), ws=None) == 3
    assert attend(shape(), ws=ODD) == 1


def test_commit_refuses():
    assert commit(None) == 1
    for name in ("tau", "acc", "table", "ctx", "kc", "vc", "out"):
        assert commit(shape(), **{name: None}) == 1, name
    for name in ("kc", "vc"):
        assert commit(shape(), **{name: ODD}) == 1, name
    assert commit(shape(), layers=0) == 1
    assert commit(shape(), layers=1025) == 1
    assert commit(shape(), B=0) == 1
    assert commit(shape(), B=8193) == 1
    assert commit(shape(), stride=10 * 2 * 16 * 64 - 8) == 1
    assert commit(shape(), stride=10 * 2 * 16 * 64 + 4) == 1
    assert commit(shape(), ctx=C.c_void_p(4096), out=C.c_void_p(4100)) == 1
    assert commit(shape(), ctx=C.c_void_p(4100), out=C.c_void_p(4096)) == 1


def test_binding_checks_tensors():
    t = torch.zeros(4, 6, dtype=torch.int32)
    cpu = -1  # the device index of host tensors
    assert pct._want("t", t, torch.int32, (4, 6), cpu) == t.data_ptr()
    for bad in (t.long(), t[:, :5], t.T, t[:3]):
        with pytest.raises(ValueError):
            pct._want("t", bad, torch.int32, (4, 6), cpu)
    with pytest.raises(ValueError):
        pct._want("t", t, torch.int32, (4, 6), 0)
    x = torch.zeros(2, 3, 10, 16, dtype=torch.bfloat16)
    s = (2, 3, 4, 16)
    assert pct._rows("x", x[:, :, 2:6], x.dtype, s, cpu)[1] == 160
    assert pct._rows("x", x[:, :, :4].contiguous(), x.dtype, s, cpu)[1] == 64
    one = x[:, :1, :4]
    assert pct._rows("x", one, x.dtype, (2, 1, 4, 16), cpu)[1] == 480
    assert pct._rows("x", x[:1, :1, :4], x.dtype, (1, 1, 4, 16), cpu)[1] == 64
    for bad in (x[:, :, :4].float(), x[:, :, :5], x[:, :, ::2][:, :, :4],
                x[:, :, :4].transpose(2, 3).contiguous().transpose(2, 3),
                torch.zeros(3, 2, 4, 16, dtype=x.dtype).transpose(0, 1),
                torch.zeros(2, 5, 4, 16, dtype=x.dtype)[:, :3]):
        with pytest.raises(ValueError):
            pct._rows("x", bad, x.dtype, s, cpu)
    with pytest.raises(ValueError):
        pct._rows("x", x[:, :, :4], x.dtype, s, 0)
    with pytest.raises(ValueError):
        pct._cache_dtype(torch.float32)
    # host tensors are refused before any call
    c = torch.zeros(3, 2, 8, 16, dtype=torch.bfloat16)
    i = torch.zeros(2, 1, dtype=torch.int64)
    with pytest.raises(ValueError):
        pct.cache_write(c, c, i, c, c)
    j = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pct.cache_commit(j[:, 0], j, j[:, 0], None, j, c, c)


def test_definition_of_the_plan():
    table = np.full((2, 3), -1, np.int32)
    (table, held, ring, state), (slot, pos, missing) = cacheref.plan(
        np.array([3, 0]), np.array([1, -1]), 2, 4, table,
        np.zeros(2, np.int32), np.array([5, 2, 7, 0], np.int32),
        np.array([3, 4], np.int32), np.array([[1, 2], [1, 1]]))
    assert table.tolist() == [[0, 5, -1], [-1, -1, -1]]
    assert held.tolist() == [2, 0] and state.tolist() == [1, 2]
    assert slot.tolist() == [[3, 20, -1], [-1, -1, -1]]
    assert pos.tolist() == [[3, 4, -1], [-1, -1, -1]]
    assert missing.tolist() == [0, 0]


def test_definition_of_attention():
    c = cacheref.Case(1, 2, 6, 4, 2, 16, 4, [9, 0], n=[6, 2])
    out, lse, _, _ = c.want()
    t = np.arange(9 + 7)
    k = c.k[c.table[0][t // 4], :, t % 4].double()
    v = c.v[c.table[0][t // 4], :, t % 4].double()
    for i in range(7):
        see = [x for x in t if x <= 9 or (i > 0 and c.anc[0, i - 1, x - 10])]
        for h in range(4):
            z = k[see, h // 2] @ c.q[0, i, h].double() * c.scale
            want = torch.softmax(z, 0) @ v[see, h // 2]
            assert np.allclose(out[0, i, h], want.numpy(), atol=1e-13)
            assert abs(lse[0, i, h] - float(torch.logsumexp(z, 0))) < 1e-13
    assert np.isnan(out[1, 3:]).all() and np.isfinite(out[1, :3]).all()
