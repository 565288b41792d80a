"""CPU checks of the rotary calls: the table of frequencies against its
definition, and the refusal of bad arguments before anything is enqueued."""
import ctypes as C
import math

import numpy as np
import pytest

import draft_tree_construction_markov_amd as pct
from rotaryref import turns
from test_cache_abi import D, HEADS, ODD, PAGES, shape


def desc(**kw):
    d = dict(rot=64, layout=0, scaling=0, original=4096, base=10000.0,
             factor=4.0, low=1.0, high=4.0, amplitude=1.0)
    d.update(kw)
    return pct.RotaryDesc(**d)


def table(d):
    out = (C.c_uint64 * max(d.rot // 2, 1))()
    rc = pct.lib().pct_rotary_table(C.byref(d), out)
    return rc, np.array([int(x) for x in out], dtype=object)


@pytest.mark.parametrize("rot", [2, 4, 18, 64, 128, 256])
@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=4.0)), ("linear", dict(factor=0.5)),
    ("base", dict(factor=8.0)),
    ("ramp", dict(factor=16.0, original=8192, low=1.0, high=32.0)),
    ("ramp", dict(factor=2.0, original=1, low=1.0, high=32.0)),
    ("bands", dict(factor=8.0, original=8192)),
    ("bands", dict(factor=8.0, original=300, low=0.25, high=7.0))])
@pytest.mark.parametrize("base", [1.5, 10000.0, 500000.0])
def test_table(rot, scaling, kw, base):
    if scaling == "base" and rot == 2:
        pytest.skip("no such scaling")
    rc, got = table(desc(rot=rot, base=base,
                         scaling=pct.Rotary.SCALINGS.index(scaling), **kw))
    assert rc == 0
    want = turns(rot, base=base, scaling=scaling, **kw)
    # the definition's own powers and logarithms are good to a few 2^-53
    for g, w in zip(got, want):
        assert abs(g / 2.0 ** 64 - w % 1.0) <= 64 * 2.0 ** -53 * max(w, 1e-3), (
            g, w)


def test_table_of_whole_turns_wraps():
    # one radian per position over a factor that makes it 1 + 1/4 turns
    rc, got = table(desc(rot=2, scaling=1, factor=1 / (2.5 * math.pi)))
    assert rc == 0
    assert abs(got[0] / 2.0 ** 64 - 0.25) < 1e-14


@pytest.mark.parametrize("bad", [
    dict(rot=-2), dict(rot=3), dict(rot=258), dict(layout=2), dict(layout=-1),
    dict(scaling=5), dict(scaling=-1), dict(base=1.0), dict(base=math.nan),
    dict(base=math.inf), dict(scaling=1, factor=0.0),
    dict(scaling=1, factor=-1.0), dict(scaling=2, factor=math.nan),
    dict(scaling=2, rot=2), dict(scaling=3, original=0),
    dict(scaling=4, low=0.0), dict(scaling=4, high=1.0),
    dict(scaling=3, high=math.inf), dict(amplitude=math.nan),
    dict(amplitude=1e39)])
def test_table_refuses(bad):
    assert table(desc(**bad))[0] == 1
    assert pct.lib().pct_last_error()


def test_table_refuses_null():
    assert pct.lib().pct_rotary_table(None, None) == 1
    assert pct.lib().pct_rotary_table(C.byref(desc()), None) == 1
    assert pct.lib().pct_rotary_table(C.byref(desc(rot=0)), None) == 0


FAR = 1 << 24


def write(sh, d=desc(), eps=1e-6, qs=256, ks=128, vs=128, os=256, **kw):
    a = dict(table=D, qw=None, kw=None, q=D, k=C.c_void_p(FAR),
             v=C.c_void_p(2 * FAR), pos=D, slot=D, out=C.c_void_p(3 * FAR),
             kc=D, vc=D)
    a.update(kw)
    return pct.lib().pct_cache_write_rotary(
        None if sh is None else C.byref(sh), None if d is None else C.byref(d),
        a["table"], eps, a["qw"], a["kw"], a["q"], qs, a["k"], ks, a["v"], vs,
        a["pos"], a["slot"], a["out"], os, a["kc"], a["vc"], None)


@pytest.mark.parametrize("bad", [p for p in PAGES if "max_pages" not in p]
                         + HEADS + [dict(Hq=5), dict(Hq=0),
                                    dict(Hq=2048, Hkv=2)])
def test_write_checks_sizes(bad):
    assert write(shape(**bad), qs=1 << 20, ks=1 << 20, vs=1 << 20,
                 os=1 << 20) == 1


def test_write_refuses():
    assert write(None) == 1
    assert write(shape(), d=None) == 1
    for name in ("table", "q", "k", "v", "pos", "slot", "out", "kc", "vc"):
        assert write(shape(), **{name: None}) == 1, name
    for name in ("q", "k", "v", "out", "kc", "vc"):
        assert write(shape(), **{name: ODD}) == 1, name
    assert write(shape(), q=None, out=None, k=None, v=None) == 1
    for name in ("qs", "ks", "vs", "os"):
        assert write(shape(), **{name: 120 if name[0] in "kv" else 248}) == 1
        assert write(shape(), **{name: 132 if name[0] in "kv" else 260}) == 1
    for eps in (-1e-6, math.nan, math.inf):
        assert write(shape(), eps=eps) == 1
    for d in (desc(rot=66), desc(rot=3), desc(layout=4),
              desc(amplitude=math.inf)):
        assert write(shape(), d=d) == 1
    assert write(shape(batch=65536)) == 2


def test_write_refuses_an_output_that_overlaps():
    rows = 2 * 9
    end = 256 + 2 * (rows * 256)
    assert write(shape(), out=C.c_void_p(end - 16)) == 1
    assert write(shape(), out=D, os=264) == 1
    assert write(shape(), out=C.c_void_p(FAR + 16)) == 1
    assert write(shape(), out=C.c_void_p(2 * FAR - 16)) == 1


def test_write_does_not_read_the_table_width():
    # a refusal that comes after the sizes' checks
    for width in (0, -1, 1 << 27, 2 ** 31 - 1):
        assert write(shape(max_pages=width), eps=-1.0) == 1
        assert b"eps" in pct.lib().pct_last_error(), width
    for heads in (0, -1, 5, 2 ** 31 - 1):
        assert write(shape(Hq=heads), q=None, out=None, eps=-1.0) == 1
        assert b"eps" in pct.lib().pct_last_error(), heads
