"""GPU checks of the rows' norm and rotation on their way into the paged cache
against the 64-bit definition."""
import numpy as np
import pytest
import torch

import draft_tree_construction_markov_amd as pct
from gpu_util import announce, dev_i32
from rotaryref import rotate, tolerance

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
SCALED = {"none": {}, "linear": dict(factor=3.0), "base": dict(factor=8.0),
          "ramp": dict(factor=16.0, original=4096),
          "bands": dict(factor=8.0, original=4096)}


class Case:
    def __init__(self, batch, N, Hq, Hkv, D, page, rot, layout, scaling, norm,
                 dtype, far=False, seed=0, unused=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        R = N + 1
        self.batch, self.R, self.Hq, self.Hkv, self.D = batch, R, Hq, Hkv, D
        self.page, self.P = page, 2 + -(-batch * R // page) * 2
        self.dtype, self.eps = dtype, 1e-5
        self.qkv = (2.0 * torch.randn(batch, R, Hq + 2 * Hkv, D, generator=g)
                    ).to(dtype).cuda()
        self.q = self.qkv[:, :, :Hq]
        self.k = self.qkv[:, :, Hq:Hq + Hkv]
        self.v = self.qkv[:, :, Hq + Hkv:]
        pos = rng.integers(0, 2 ** 30 if far else 5000, (batch, R))
        pos.flat[0] = 2 ** 30 if far else 0
        slot = rng.permutation(self.P * page)[:batch * R].reshape(batch, R)
        if unused:
            pos[rng.random((batch, R)) < 0.2] = -1
            slot[rng.random((batch, R)) < 0.2] = -1
            slot.flat[-1] = self.P * page
        self.pos, self.slot = pos, slot
        self.w = [1.0 + 0.5 * torch.randn(D, generator=g) if norm else None
                  for _ in range(2)]
        self.rotary = pct.Rotary(D, rot=rot, layout=layout, scaling=scaling,
                                 **SCALED[scaling])
        self.cache = [torch.randn(self.P, Hkv, page, D, generator=g).to(
            dtype).cuda() for _ in range(2)]
        self.before = [c.clone() for c in self.cache]
        self.out = torch.randn(batch, R, Hq, D, generator=g).to(dtype).cuda()
        self.was = self.out.clone()

    def dev(self):
        return (dev_i32(self.pos),
                torch.from_numpy(self.slot.astype(np.int64)).cuda())

    def call(self, q=True, kv=True, out=None):
        pos, slot = self.dev()
        w = [None if x is None else x.cuda() for x in self.w]
        return pct.cache_write_rotary(
            self.rotary, self.q if q else None, self.k if kv else None,
            self.v if kv else None, pos, slot, *self.cache, q_weight=w[0],
            k_weight=w[1], eps=self.eps, out=self.out if out is None else out)

    def want(self, x, weight):
        d = self.rotary.desc
        f = [int(v) % (1 << 64) for v in self.rotary.table.cpu().tolist()]
        y, mag = rotate(x.float().cpu().numpy(), np.maximum(self.pos, 0), f,
                        d.rot, pct.Rotary.LAYOUTS[d.layout], d.amplitude,
                        None if weight is None else weight.double().numpy(),
                        self.eps)
        return y, tolerance(y, mag, self.dtype)

    def check_q(self, got, was, q):
        y, tol = self.want(q, self.w[0])
        on = self.pos >= 0
        got_ = got.float().cpu().numpy()
        err = np.abs(got_ - y)
        assert (err[on] <= tol[on]).all(), float((err - tol)[on].max())
        assert np.array_equal(got_[~on], was.float().cpu().numpy()[~on])

    def check_cache(self, k, v):
        y, tol = self.want(k, self.w[1])
        want_v = self.before[1].clone()
        got = self.cache[0].float().cpu().numpy()
        left = np.ones((self.P, self.page), bool)
        for b in range(self.batch):
            for i in range(self.R):
                s = int(self.slot[b, i])
                if s < 0 or s >= self.P * self.page or self.pos[b, i] < 0:
                    continue
                p, o = divmod(s, self.page)
                left[p, o] = False
                err = np.abs(got[p, :, o] - y[b, i])
                assert (err <= tol[b, i]).all(), (b, i)
                want_v[p, :, o] = v[b, i]
        was = self.before[0].float().cpu().numpy()
        assert np.array_equal(got.transpose(0, 2, 1, 3)[left],
                              was.transpose(0, 2, 1, 3)[left])
        assert torch.equal(self.cache[1].view(torch.int16),
                           want_v.view(torch.int16))


CASES = [
    # batch N Hq Hkv D page rot layout scaling norm type far
    (1, 0, 32, 8, 128, 16, 128, "half", "none", True, BF, False),
    (1, 0, 1, 1, 16, 1, 16, "half", "none", False, HF, False),
    (3, 7, 4, 2, 64, 16, 64, "half", "linear", True, HF, True),
    (3, 7, 4, 2, 64, 16, 64, "interleaved", "base", True, BF, True),
    (2, 33, 14, 2, 80, 64, 40, "interleaved", "ramp", False, HF, True),
    (2, 33, 14, 2, 80, 64, 20, "half", "ramp", True, BF, False),
    (5, 4, 7, 7, 96, 8, 24, "half", "bands", True, HF, True),
    (5, 4, 6, 3, 96, 8, 96, "half", "bands", False, BF, True),
    (2, 20, 16, 1, 112, 32, 112, "half", "none", True, HF, False),
    (2, 20, 16, 1, 256, 32, 256, "half", "none", True, BF, True),
    (4, 3, 8, 8, 192, 4, 64, "interleaved", "linear", True, HF, False),
    (4, 3, 8, 4, 176, 4, 176, "half", "none", False, BF, False),
    (6, 2, 5, 5, 32, 16, 2, "half", "none", True, HF, True),
    (6, 2, 5, 5, 32, 16, 6, "interleaved", "none", False, BF, True),
    (6, 2, 10, 5, 48, 128, 0, "half", "none", True, HF, False),
    (6, 2, 10, 5, 240, 128, 14, "half", "ramp", True, HF, True),
    (128, 63, 8, 2, 64, 16, 64, "half", "bands", True, BF, False),
    (70, 300, 2, 1, 32, 32, 32, "half", "none", True, HF, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rotary(case):
    c = Case(*case)
    q, k, v = c.q.clone(), c.k.clone(), c.v.clone()
    announce("rotary", case)
    got = c.call()
    torch.cuda.synchronize()
    assert got is c.out
    c.check_q(got, c.was, q)
    c.check_cache(k, v)
    assert torch.equal(c.q, q) and torch.equal(c.k, k)


@pytest.mark.parametrize("case", [CASES[4], CASES[5], CASES[10]],
                         ids=["pairs", "odd", "wide"])
def test_in_place(case):
    c = Case(*case, seed=3)
    q, k, v = c.q.clone(), c.k.clone(), c.v.clone()
    announce("rotary in place", case)
    got = c.call(out=c.q)
    torch.cuda.synchronize()
    c.check_q(got, q, q)
    c.check_cache(k, v)
    assert torch.equal(c.k, k) and torch.equal(c.v, v)


def test_queries_or_keys_alone():
    c = Case(*CASES[2], seed=4)
    announce("rotary, queries alone")
    got = c.call(kv=False)
    torch.cuda.synchronize()
    c.check_q(got, c.was, c.q)
    assert all(torch.equal(x, y) for x, y in zip(c.cache, c.before))
    announce("rotary, keys and values alone")
    assert c.call(q=False) is None
    torch.cuda.synchronize()
    c.check_cache(c.k, c.v)


def test_what_is_not_finite_stays_in_its_pair_or_head():
    c = Case(2, 3, 4, 2, 64, 16, 32, "half", "none", False, BF, unused=False)
    c.q[0, 1, 2, 3] = float("nan")
    c.q[1, 0, 0, 40] = float("inf")   # not rotated
    c.v[0, 0, 0, :4] = torch.tensor([float("nan"), float("inf"), -0.0, 0.0],
                                    dtype=BF)
    q = c.q.clone()
    announce("rotary, not finite")
    got = c.call()
    torch.cuda.synchronize()
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 1, 2, 3] = bad[0, 1, 2, 3 + 16] = True
    assert torch.equal(got.isnan(), bad)
    assert got[1, 0, 0, 40] == float("inf")
    q[0, 1, 2, 3], q[1, 0, 0, 40] = 0.0, 0.0
    y, tol = c.want(q, None)
    ok = ~(bad | got.isinf()).cpu().numpy()
    assert (np.abs(got.float().cpu().numpy() - y)[ok] <= tol[ok]).all()
    c.check_cache(c.k, c.v)


def test_heads_of_zeros():
    c = Case(1, 2, 4, 2, 64, 16, 64, "half", "none", True, HF, unused=False)
    c.qkv.zero_()
    announce("rotary, zeros")
    got = c.call()
    torch.cuda.synchronize()
    assert not got.any()
    c.check_cache(c.k, c.v)


def test_other_stream_and_graph():
    c = Case(3, 7, 8, 2, 128, 16, 128, "half", "none", True, BF, seed=5,
             unused=False)
    pos, slot = c.dev()
    w = [x.cuda() for x in c.w]

    def call():
        return pct.cache_write_rotary(c.rotary, c.q, c.k, c.v, pos, slot,
                                      *c.cache, q_weight=w[0], k_weight=w[1],
                                      eps=c.eps, out=c.out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    announce("rotary, other stream")
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    c.check_q(c.out, c.was, c.q)
    announce("rotary, graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for turn in range(3):
        c.qkv.normal_()
        c.pos = (c.pos + 977) % 4000
        pos.copy_(dev_i32(c.pos))
        c.before = [x.clone() for x in c.cache]
        g.replay()
        torch.cuda.synchronize()
        c.check_q(c.out, c.was, c.q)
        c.check_cache(c.k, c.v)


def test_binding_refuses():
    c = Case(*CASES[2], seed=6)
    pos, slot = c.dev()
    ok = (c.rotary, c.q, c.k, c.v, pos, slot, *c.cache)

    def bad(at, x):
        args = list(ok)
        args[at] = x
        with pytest.raises(ValueError):
            pct.cache_write_rotary(*args)

    bad(0, pct.Rotary(32))
    bad(1, c.q[:, :, :, ::2])
    bad(1, c.q.float())
    bad(2, None)
    bad(2, c.k.cpu())
    bad(4, pos.long())
    bad(5, slot.int())
    bad(5, slot[:, :-1])
    bad(7, c.cache[1][:1])
    with pytest.raises(ValueError):
        pct.cache_write_rotary(*ok, q_weight=torch.ones(
            64, dtype=HF, device="cuda"))
    with pytest.raises(pct.PCTError):
        pct.cache_write_rotary(*ok, out=c.qkv[:, :, 1:5])
    for kw in (dict(layout="x"), dict(scaling="x"), dict(rot=66)):
        with pytest.raises(ValueError):
            pct.Rotary(64, **kw)
    with pytest.raises(pct.PCTError):
        pct.Rotary(64, scaling="ramp", factor=2.0)


def test_a_round_of_the_cache():
    torch.manual_seed(0)
    N, Hq, Hkv, D = 3, 4, 2, 64
    c = pct.PagedCache(2, N, 12, 4, 6, Hq, Hkv, D, layers=2)
    c.ctx_len.copy_(torch.tensor([5, 0]))
    depth = dev_i32([[1, 2, 2], [1, 1, 0]])
    rows = c.plan(dev_i32([3, 2]), depth)
    r = pct.Rotary(D)
    qkv = torch.randn(2, N + 1, Hq + 2 * Hkv, D, device="cuda").bfloat16()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    announce("rotary, a round")
    out = c.write_rotary(1, r, q, k, v)
    torch.cuda.synchronize()
    f = [int(x) % (1 << 64) for x in r.table.tolist()]
    pos = rows.pos.cpu().numpy()
    assert pos.tolist() == [[5, 6, 7, 7], [0, 1, 1, -1]]
    for x, got in ((q, lambda b, i: out[b, i]),
                   (k, lambda b, i: c.k[1, rows.slot[b, i] // 4, :,
                                        rows.slot[b, i] % 4])):
        y, mag = rotate(x.float().cpu().numpy(), np.maximum(pos, 0), f, D,
                        "half")
        tol = tolerance(y, mag, BF)
        for b in range(2):
            for i in range(N + 1):
                if pos[b, i] >= 0:
                    err = np.abs(got(b, i).float().cpu().numpy() - y[b, i])
                    assert (err <= tol[b, i]).all()
    assert not out[1, 3].any() and not c.k[0].any()


@pytest.mark.parametrize("power", [-100, -60, 45, 100])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_squares_past_the_range_of_fp32(power, eps):
    c = Case(2, 5, 4, 2, 80, 16, 80, "half", "none", True, BF, unused=False)
    c.qkv.mul_(2.0 ** power)
    c.qkv[0, 1] = 1.0
    c.eps = eps
    q, k, v = c.q.clone(), c.k.clone(), c.v.clone()
    announce("rotary, powers", power, eps)
    got = c.call()
    torch.cuda.synchronize()
    c.check_q(got, c.was, q)
    c.check_cache(k, v)


def test_more_rows_than_a_grid_has_threads_for():
    # 2^26 + 8193 rows of one head of 16 elements, in place: rows on both sides
    # of every 2^24th one, the first and the last against the definition
    R, batch, D = 8193, 8193, 16
    rows = R * batch
    assert rows > 1 << 26
    rotary = pct.Rotary(D)
    cache = torch.zeros(1, 1, 1, D, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn(rows, D, generator=g, device="cuda", dtype=BF)
    q = q.view(batch, R, 1, D)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    pos[rows - 2] = -1
    at = sorted({x for m in range(0, rows, 1 << 24) for x in (m, m - 1)
                 if x >= 0} | {rows - 1, rows - 2, rows - 8193, 1 << 26})
    was = q.view(rows, D)[at].float().cpu().numpy()
    announce("rotary, rows past 2^26", rows)
    out = pct.cache_write_rotary(rotary, q, None, None, pos.view(batch, R),
                                 None, cache, cache, out=q)
    torch.cuda.synchronize()
    assert out is q
    got = q.view(rows, D)[at].float().cpu().numpy()
    f = [int(x) % (1 << 64) for x in rotary.table.cpu().tolist()]
    y, mag = rotate(was[:, None], np.array(at), f, D, "half")
    tol = tolerance(y, mag, BF)
    for i, x in enumerate(at):
        if x == rows - 2:
            assert np.array_equal(got[i], was[i])
        else:
            assert (np.abs(got[i] - y[i, 0]) <= tol[i, 0]).all(), x
            assert x == 0 or not np.array_equal(got[i], was[i]), x
