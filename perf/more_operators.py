"""Measured cases of shared and rotated rows on a paged key-value cache: the
norm and position rotation of a round's queries and keys on their way into the
cache, the plan of which requests share a prefix, attention that reads a
shared prefix once for all of its requests, and the cache's pages as requests
fork, end and are moved together.

Positions and rows are those of perf/operators.py: a request's cache positions
are its ctx_len committed tokens, its root and its drafted nodes; row 0 of a
request is the root, row 1 + i is node i, n_nodes = -1 marks a padded request.

own = False computes the operators from elementary torch operations, own =
True with the package's calls.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one new token of one request: the latency of a chat's decoding step
        dict(name="rotary, one token", op="rotary", batch=1, N=0, Hq=32,
             Hkv=8, D=128, page=16, rot=128, layout="half", scaling="none",
             norm=True, type="bf16", full=True, ctx_hi=4001),
        # straight drafts at far positions, part of each head rotated in
        # neighbouring pairs, frequencies scaled by a ramp, half precision,
        # one padded request
        dict(name="rotary, chains, fp16", op="rotary", batch=33, N=16, Hq=14,
             Hkv=2, D=80, page=64, rot=40, layout="interleaved",
             scaling="ramp", norm=False, type="fp16", full=False,
             ctx_hi=900001),
        # the rows of the round workload's trees
        dict(name="rotary, trees, batch 128", op="rotary", batch=128, N=512,
             Hq=32, Hkv=8, D=128, page=16, rot=128, layout="half",
             scaling="bands", norm=True, type="bf16", full=True,
             ctx_hi=32768),
        # who shares what among a few requests with a common prompt
        dict(name="share plan, batch 8", op="share", batch=8, N=0, page=16,
             groups=1, alone=1, prefix=1001, own_lo=3, own_hi=300),
        # a serving batch: three prompts and some requests of their own
        dict(name="share plan, batch 128", op="share", batch=128, N=7,
             page=16, groups=3, alone=9, prefix=16384, own_lo=64,
             own_hi=4096),
        # four samples of one prompt, half precision, straight drafts of
        # uneven lengths, normalisers kept
        dict(name="shared attention, 4 samples, fp16", op="attend", batch=4,
             N=5, Hq=14, Hkv=2, D=64, page=64, groups=1, alone=0,
             prefix=1001, own_lo=1, own_hi=90, type="fp16", full=False,
             chain=True),
        # plain decoding of a serving batch whose requests share one of two
        # long documents, and some requests of their own
        dict(name="shared attention, one token, batch 128", op="attend",
             batch=128, N=0, Hq=32, Hkv=8, D=128, page=16, groups=2,
             alone=5, prefix=16384, own_lo=64, own_hi=4096, type="bf16",
             full=True, chain=False),
        # the b7 workload's trees over a shared document
        dict(name="shared attention, trees, batch 16", op="attend",
             batch=16, N=64, Hq=32, Hkv=8, D=128, page=32, groups=1, alone=0,
             prefix=8200, own_lo=30, own_hi=1500, type="bf16", full=True,
             chain=False),
        # four new samples of one prompt take the place of four others
        dict(name="free and fork, 4 samples", op="fork", forks=4, sources=1,
             N=0, Hkv=8, D=128, page=16, layers=32, ctx_lo=1001, ctx_hi=1001,
             type="bf16"),
        # a step of a search with 8 candidates for each of 8 requests
        dict(name="free and fork, 64 candidates", op="fork", forks=64,
             sources=8, N=64, Hkv=8, D=128, page=32, layers=16, ctx_lo=505,
             ctx_hi=4090, type="bf16"),
        # the cache after half of its requests ended
        dict(name="compact, batch 4", op="compact", batch=4, Hkv=8, D=128,
             page=16, layers=4, ctx_lo=100, ctx_hi=900, used=0.5,
             type="bf16"),
        # a large cache of which a third is in use
        dict(name="compact, batch 64", op="compact", batch=64, Hkv=8, D=128,
             page=16, layers=16, ctx_lo=64, ctx_hi=1800, used=0.35,
             type="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(
        math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary"] * 3 + ["share"] * 2 + ["attend"] * 5
                    + ["fork", "compact"])
    c = dict(op=op, page=rng.choice([8, 16, 32, 64, 128]))
    if op == "share":
        c.update(batch=_log_int(rng, 2, 128), N=rng.randint(0, 64),
                 prefix=_log_int(rng, 16, 16384), own_lo=_log_int(rng, 1, 64),
                 own_hi=_log_int(rng, 64, 4096))
        c["groups"] = rng.randint(1, max(1, min(6, c["batch"] // 2)))
        c["alone"] = rng.randint(0, c["batch"] - 2 * c["groups"])
        return c
    c.update(Hkv=rng.choice([1, 2, 4, 8]),
             D=rng.choice([64, 80, 96, 128, 192, 256]),
             type=rng.choice(["bf16", "fp16"]))
    if op == "fork":
        c.update(forks=_log_int(rng, 1, 64), N=rng.randint(0, 64),
                 layers=rng.randint(1, 16), ctx_lo=_log_int(rng, 1, 512),
                 ctx_hi=_log_int(rng, 512, 4096))
        c["sources"] = rng.randint(1, min(8, c["forks"]))
        return _small_cache(c, c["sources"], 64 * 0.5 * c["page"] * c["forks"])
    if op == "compact":
        c.update(batch=_log_int(rng, 1, 64), layers=rng.randint(1, 16),
                 ctx_lo=_log_int(rng, 1, 128), ctx_hi=_log_int(rng, 128, 1800),
                 used=rng.uniform(0.2, 0.9))
        return _small_cache(c, c["batch"], 0)
    c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 7, 8])
    c["full"] = rng.random() < 0.5
    if op == "rotary":
        c.update(batch=_log_int(rng, 1, 128), N=_log_int(rng, 1, 512) - 1,
                 rot=rng.choice([c["D"], c["D"] // 2, c["D"] // 4]),
                 layout=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "base", "ramp",
                                     "bands"]),
                 norm=rng.random() < 0.6, ctx_hi=_log_int(rng, 512, 1000000))
        while c["batch"] * (c["N"] + 1) * (c["Hq"] + 2 * c["Hkv"]) * c["D"] \
                > 128 * 513 * 48 * 128:
            c["batch"] = max(1, c["batch"] // 2)
            c["N"] = c["N"] * 3 // 4
        return c
    c.update(batch=_log_int(rng, 2, 128),
             N=0 if rng.random() < 0.5 else _log_int(rng, 1, 64),
             prefix=_log_int(rng, 64, 32768), own_lo=_log_int(rng, 1, 64),
             own_hi=_log_int(rng, 64, 4096), chain=rng.random() < 0.3)
    # no more cache, nor more scores, than the listed cases have
    while (c["batch"] * (c["prefix"] + c["own_hi"]) * c["Hkv"] * c["D"]
           > 128 * 20480 * 1024
           or c["batch"] * (c["N"] + 1) * c["Hq"]
           * (c["prefix"] + c["own_hi"]) > 16 * 65 * 32 * 9700):
        if c["batch"] > 8 and rng.random() < 0.5:
            c["batch"] = c["batch"] // 2
        elif c["prefix"] > 512:
            c["prefix"] = c["prefix"] * 2 // 3
        elif c["own_hi"] > 128:
            c["own_hi"] = max(c["own_lo"], c["own_hi"] // 2)
        else:
            c["batch"] = max(2, c["batch"] // 2)
            c["N"] = c["N"] // 2
    c["groups"] = rng.randint(1, max(1, min(4, c["batch"] // 2)))
    c["alone"] = rng.randint(0, (c["batch"] - 2 * c["groups"]) // 2)
    return c


def _small_cache(c, requests, more):
    """Fewer layers where the cache would be larger than the listed ones."""
    while c["layers"] > 1 and c["layers"] * c["Hkv"] * c["D"] * (
            requests * c["ctx_hi"] / c.get("used", 1.0) + more) \
            > 16 * 1024 * 64 * 1800 / 0.35 / 2:
        c["layers"] -= 1
    while requests * c["ctx_hi"] * c["Hkv"] * c["D"] / c.get("used", 1.0) \
            > 16 * 1024 * 64 * 1800 / 0.35 / 2:
        c["ctx_hi"] = max(c["ctx_lo"], c["ctx_hi"] // 2)
        if c["ctx_hi"] == c["ctx_lo"]:
            c["Hkv"] = 1
            break
    return c


def _spread(lo, hi, count):
    """`count` log-uniform quantiles of lo .. hi."""
    f = (np.arange(count) + 0.5) / count
    return np.rint(np.exp(math.log(lo) + f * (
        math.log(hi) - math.log(lo)))).astype(np.int64)


def _nodes(c):
    """Drafted nodes of the requests; they belong to the case."""
    n = np.full(c["batch"], c["N"], np.int64)
    if not c.get("full", True):
        n = c["N"] // 4 + (np.arange(c["batch"]) * 7919) % (
            c["N"] - c["N"] // 4 + 1)
        if c["batch"] >= 5:
            n[c["batch"] // 2] = -1
    return n


def _groups(c):
    """Prompt of each request (0 .. groups - 1, or -1: one of its own) and
    the lengths of the prompt and of what the request added to it."""
    i = np.arange(c["batch"])
    of = np.where(i < c["alone"], -1, i % c["groups"])
    prefix = c["prefix"] - (c["prefix"] // 5) * (of > 0) * of // max(
        1, c["groups"])
    more = _spread(c["own_lo"], c["own_hi"], c["batch"])
    return of, prefix, more[(i * 7) % c["batch"]] if c["batch"] % 7 else more


def _shared_work(c):
    """Positions read once for all, and by each request."""
    of, prefix, more = _groups(c)
    n = _nodes(c)
    once, each = 0, 0
    for g in range(-1, c["groups"]):
        on = (of == g) & (n >= 0)
        if g < 0 or on.sum() < 2:
            each += int((prefix + more + n + 1)[on].sum())
        else:
            full = int(prefix[on][0]) // c["page"] * c["page"]
            once += full
            each += int((prefix + more + n + 1 - full)[on].sum())
    return once, each


def _compact_sizes(c):
    """Context lengths, pages in use, pages of the cache."""
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])
    used = int((-(-(ctx + 1) // c["page"])).sum())
    return ctx, used, max(used + 1, int(used / c["used"]))


def work(c):
    if c["op"] == "rotary":
        rows = float((_nodes(c) + 1).sum())
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": rows * (4.0 * heads * c["D"] + 12.0),
                "flops": rows * (c["Hq"] + c["Hkv"]) * (
                    3.0 * c["rot"] + (4.0 * c["D"] if c["norm"] else 0.0))}
    if c["op"] == "share":
        of, prefix, more = _groups(c)
        return {"bytes": float(4 * ((prefix + more) // c["page"]).sum()
                               + 16 * c["batch"]), "flops": 0.0}
    if c["op"] == "fork":
        ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["sources"])
        of = np.arange(c["forks"]) % c["sources"]
        rows = float((ctx % c["page"])[of].sum())
        # each source's rows read once, each fork's written
        read = float((ctx % c["page"]).sum())
        pages = float((ctx // c["page"])[of].sum())
        return {"bytes": (rows + read) * 4.0 * c["layers"] * c["Hkv"] * c["D"]
                + 12.0 * pages, "flops": 0.0}
    if c["op"] == "compact":
        ctx, used, total = _compact_sizes(c)
        moves = used * (1.0 - used / total)  # expected, of random pages
        return {"bytes": moves * 8.0 * c["layers"] * c["Hkv"] * c["page"]
                * c["D"] + 12.0 * total + 8.0 * used, "flops": 0.0}
    once, each = _shared_work(c)
    of, prefix, more = _groups(c)
    n = _nodes(c)
    on = n >= 0
    seen = (prefix + more)[on] + 1.0 + (
        n[on] / 2 if c["chain"] else np.minimum(n[on], 4))
    rows = (n[on] + 1.0)
    return {"bytes": 4.0 * c["Hkv"] * c["D"] * (once + each)
            + 4.0 * c["Hq"] * c["D"] * float(rows.sum()),
            "flops": float(4.0 * c["D"] * c["Hq"] * (rows * seen).sum())}


# ---------------------------------------------------------------------------
# inputs

def _tree(rng, batch, N, n, chain):
    """Random draft trees in node order: depths and packed ancestry masks."""
    depth = np.zeros((batch, N), np.int32)
    bits = np.zeros((batch, N, -(-N // 64) * 64), bool)
    for i in range(N):
        p = np.full(batch, i - 1) if chain else np.floor(
            (i + 1) * rng.random(batch)).astype(np.int64) - 1
        depth[:, i] = 1
        q = np.nonzero(p >= 0)[0]
        depth[q, i] = depth[q, p[q]] + 1
        bits[q, i] = bits[q, p[q]]
        bits[:, i, i] = True
    live = np.arange(N)[None] < n[:, None]
    depth[~live], bits[~live] = 0, False
    words = np.packbits(bits, axis=2, bitorder="little").view(np.int64)
    return depth, words


def _normal(g, shape, dtype, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    x.normal_(0.0, scale, generator=g)
    return x


def _dev(a, dtype=None):
    a = np.ascontiguousarray(a if dtype is None else a.astype(dtype))
    return torch.from_numpy(a).cuda()


def _shared_table(rng, c, ctx, n, of, prefix, width):
    """Block table of requests whose prompts share their whole pages."""
    page = c["page"]
    need = -(-(ctx + n + 1) // page)
    shared = np.where(of >= 0, prefix // page, 0)
    first = {g: np.nonzero(of == g)[0][0] for g in range(c["groups"])
             if (of == g).any()}
    total = int((need - shared).sum()) + 3 + sum(
        int(shared[b]) for b in first.values())
    perm = rng.permutation(total)
    table = np.full((c["batch"], width), -1, np.int32)
    at = 0
    prompt = {}
    for g, b in first.items():
        prompt[g] = perm[at:at + shared[b]]
        at += shared[b]
    for b in range(c["batch"]):
        s = int(shared[b])
        if s:
            table[b, :s] = prompt[of[b]]
        table[b, s:need[b]] = perm[at:at + need[b] - s]
        at += need[b] - s
    return table, total


SCALING = {"none": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0),
           "ramp": dict(factor=16.0, original=8192),
           "bands": dict(factor=8.0, original=8192)}
BASE = 500000.0
EPS = 1e-6


def prepare(c, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(c)
    return {"rotary": _prepare_rotary, "share": _prepare_share,
            "attend": _prepare_attend, "fork": _prepare_fork,
            "compact": _prepare_compact}[c["op"]](c, s, rng, g)


def _prepare_rotary(c, s, rng, g):
    batch, N, page, D = c["batch"], c["N"], c["page"], c["D"]
    Hq, Hkv, dtype = c["Hq"], c["Hkv"], TYPES[c["type"]]
    n = _nodes(c)[rng.permutation(batch)]
    ctx = rng.integers(0, c["ctx_hi"], batch)
    depth = _tree(rng, min(batch, 4), N, np.full(min(batch, 4), N), False)[0]
    i = np.arange(N + 1)[None]
    pos = ctx[:, None] + np.concatenate(
        [np.zeros((batch, 1), np.int64), np.resize(depth, (batch, N))], 1)
    pos = np.where(i <= n[:, None], pos, -1)
    # the rows' places in pages of their own
    off = ctx % page
    width = -(-(page + N + 1) // page)
    table = rng.permutation(batch * width + 2)[:batch * width].reshape(
        batch, width)
    at = off[:, None] + i
    slot = table[np.arange(batch)[:, None], at // page] * page + at % page
    slot = np.where(i <= n[:, None], slot, -1)
    total = batch * width + 3
    qkv = _normal(g, (batch, N + 1, Hq + 2 * Hkv, D), dtype)
    weight = lambda: (1.0 + 0.3 * torch.randn(  # noqa: E731
        D, generator=g, device="cuda")) if c["norm"] else None
    s.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv],
             v=qkv[:, :, Hq + Hkv:], pos=_dev(pos, np.int32),
             slot=_dev(slot, np.int64), q_weight=weight(), k_weight=weight(),
             k_cache=_normal(g, (total, Hkv, page, D), dtype),
             v_cache=_normal(g, (total, Hkv, page, D), dtype),
             out=torch.zeros(batch, N + 1, Hq, D, dtype=dtype, device="cuda"))
    if own:
        import draft_tree_construction_markov_amd as pct
        s["rotary"] = pct.Rotary(D, rot=c["rot"], base=BASE,
                                 layout=c["layout"], scaling=c["scaling"],
                                 **SCALING[c["scaling"]])
    else:
        f, s["amplitude"] = _frequencies(c)
        s["frequency"] = f.cuda()
    return s


def _prepare_share(c, s, rng, g):
    of, prefix, more = _groups(c)
    order = rng.permutation(c["batch"])
    of, prefix, more, n = of[order], prefix[order], more[order], _nodes(c)
    ctx = prefix + more
    width = -(-int(ctx.max() + c["N"] + 9) // c["page"])
    table, total = _shared_table(rng, c, ctx, n, of, prefix, width)
    s.update(ctx=_dev(ctx, np.int32), n=_dev(n, np.int32), table=_dev(table),
             width=width, n_pages=total, least=512)
    if own:
        import draft_tree_construction_markov_amd as pct
        s["handle"] = pct.SharePlan(c["batch"], c["N"], total, c["page"],
                                    width, least=s["least"])
    return s


def _prepare_attend(c, s, rng, g):
    batch, N, page, D = c["batch"], c["N"], c["page"], c["D"]
    Hq, Hkv, dtype = c["Hq"], c["Hkv"], TYPES[c["type"]]
    of, prefix, more = _groups(c)
    order = rng.permutation(batch)
    of, prefix, more, n = (x[order] for x in (of, prefix, more, _nodes(c)))
    ctx = prefix + more
    width = -(-int(ctx.max() + N + 1) // page)
    table, total = _shared_table(rng, c, ctx, n, of, prefix, width)
    mask = None
    if N > 0 and not c["chain"]:
        mask = _dev(_tree(rng, batch, N, n, False)[1])
    # keys share a bias in each channel, as trained projections do
    k = _normal(g, (total, Hkv, page, D), dtype)
    k += _normal(g, (Hkv, 1, D), dtype)
    s.update(ctx=_dev(ctx, np.int32), n=_dev(n, np.int32), table=_dev(table),
             width=width, mask=mask, scale=D ** -0.5, k_cache=k,
             v_cache=_normal(g, (total, Hkv, page, D), dtype),
             q=_normal(g, (batch, N + 1, Hq + 2 * Hkv, D), dtype, 1.5)
             [:, :, :Hq])
    if own:
        import draft_tree_construction_markov_amd as pct
        # planned once for all layers of a round
        s["plan"] = pct.SharePlan(batch, N, total, page, width)
        s["share"] = s["plan"].run(s["ctx"], s["n"], s["table"])
        s["handle"] = pct.SharedAttention(batch, N, Hq, Hkv, D, total, page,
                                          width, dtype=dtype, lse=True)
    return s


def _prepare_fork(c, s, rng, g):
    """`sources` requests, each with its share of the forks, which were made
    at this length and not advanced: the pass ends them and makes them anew."""
    page, S, F = c["page"], c["sources"], c["forks"]
    batch = S + F
    ctx = np.zeros(batch, np.int64)
    ctx[:S] = _spread(c["ctx_lo"], c["ctx_hi"], S)
    place = rng.permutation(batch)  # which place of the batch is which
    of = np.arange(F) % S
    ctx[S:] = ctx[of]
    held = np.where(np.arange(batch) < S, -(-(ctx + c["N"] + 1) // page),
                    -(-ctx // page))
    width = int(held.max()) + 2
    total = int(held[:S].sum()) + 2 * F + 5
    perm = rng.permutation(total)
    table = np.full((batch, width), -1, np.int32)
    extra = np.zeros(total, np.int32)
    at = 0
    for b in range(S):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    for i in range(F):
        b, full = S + i, int(ctx[of[i]]) // page
        table[b, :full] = table[of[i], :full]
        extra[table[b, :full]] += 1
        if held[b] > full:
            table[b, full] = perm[at]
            at += 1
    free = perm[at:]
    ring = np.concatenate([free, np.full(at, -1)])
    head = int(rng.integers(total))
    out = lambda a: a[np.argsort(place)]  # noqa: E731
    src = np.concatenate([place[of], [-1]])
    dst = np.concatenate([place[S:], [-1]])
    dtype = TYPES[c["type"]]
    shape = (c["layers"], total, c["Hkv"], page, c["D"])
    s.update(batch=batch, width=width, n_pages=total,
             src=_dev(src, np.int32), dst=_dev(dst, np.int32),
             ctx=_dev(out(ctx), np.int32), held=_dev(out(held), np.int32),
             table=_dev(out(table)), extra=_dev(extra),
             ring=_dev(np.roll(ring, head), np.int32),
             ring_state=_dev(np.array([head, len(free)]), np.int32),
             k_cache=_normal(g, shape, dtype), v_cache=_normal(g, shape, dtype))
    if own:
        import draft_tree_construction_markov_amd as pct
        s["handle"] = pct.CachePages(batch, total, page, width, c["Hkv"],
                                     c["D"], layers=c["layers"], dtype=dtype)
        s["state"] = pct.PageState(s["ctx"], s["table"], s["held"], s["ring"],
                                   s["ring_state"], s["extra"])
    return s


def _prepare_compact(c, s, rng, g):
    """Requests on random pages of the cache; every fourth one shares its
    first pages with the one before it."""
    page, batch = c["page"], c["batch"]
    ctx, used, total = _compact_sizes(c)
    held = -(-(ctx + 1) // page)
    width = int(held.max()) + 1
    perm = rng.permutation(total)
    table = np.full((batch, width), -1, np.int32)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
        if b % 4 == 3:
            m = int(min(held[b - 1], held[b]) // 2)
            table[b, :m] = table[b - 1, :m]
    order = rng.permutation(batch)
    dtype = TYPES[c["type"]]
    shape = (c["layers"], total, c["Hkv"], page, c["D"])
    i32 = dict(dtype=torch.int32, device="cuda")
    s.update(n_pages=total, width=width, table=_dev(table[order]),
             held=_dev(held[order], np.int32), ctx=_dev(ctx[order], np.int32),
             table_new=torch.zeros(batch, width, **i32),
             ring=torch.zeros(total, **i32),
             ring_state=torch.zeros(2, **i32),
             extra=torch.zeros(total, **i32),
             k_cache=_normal(g, shape, dtype), v_cache=_normal(g, shape, dtype))
    if own:
        import draft_tree_construction_markov_amd as pct
        s["handle"] = pct.CachePages(batch, total, page, width, c["Hkv"],
                                     c["D"], layers=c["layers"], dtype=dtype)
        s["state"] = pct.PageState(s["ctx"], s["table"], s["held"], s["ring"],
                                   s["ring_state"], s["extra"])
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    if not own:
        return {"rotary": _rotary, "share": _share, "attend": _attend,
                "fork": _fork, "compact": _compact}[s["op"]](s)
    import draft_tree_construction_markov_amd as pct
    if s["op"] == "rotary":
        q = pct.cache_write_rotary(
            s["rotary"], s["q"], s["k"], s["v"], s["pos"], s["slot"],
            s["k_cache"], s["v_cache"], q_weight=s["q_weight"],
            k_weight=s["k_weight"], eps=EPS, out=s["out"])
        return q, s["k_cache"], s["v_cache"]
    if s["op"] == "share":
        o = s["handle"].run(s["ctx"], s["n"], s["table"])
        return o.leader, o.shared
    if s["op"] == "attend":
        return s["handle"].run(s["q"], s["k_cache"], s["v_cache"], s["table"],
                               s["share"], mask=s["mask"], scale=s["scale"])
    if s["op"] == "fork":
        s["handle"].free(s["state"], s["dst"])
        done = s["handle"].fork(s["state"], s["src"], s["dst"], s["k_cache"],
                                s["v_cache"])
        return (done, s["ctx"], s["table"], s["held"], s["ring"],
                s["ring_state"], s["extra"], s["k_cache"], s["v_cache"])
    s["handle"].compact(s["state"], s["k_cache"], s["v_cache"],
                        out=s["table_new"])
    return (s["table_new"], s["ring"], s["ring_state"], s["extra"],
            s["k_cache"], s["v_cache"])


def _frequencies(c):
    """Radians per position of each pair, in 64 bits, and the factor of the
    rotated elements."""
    rot, kind = c["rot"], c["scaling"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    par = SCALING[kind]
    f = BASE ** (-2.0 * i / rot)
    if kind == "linear":
        return f / par["factor"], 1.0
    if kind == "base":
        wide = BASE * par["factor"] ** (rot / (rot - 2.0))
        return wide ** (-2.0 * i / rot), 1.0
    if kind == "ramp":
        # the pairs that make 32 turns and one turn in the original length
        at = [rot * math.log(par["original"] / (2 * math.pi * turns))
              / (2 * math.log(BASE)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        w = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return (f * (1.0 - w) + f / par["factor"] * w,
                1.0 + 0.1 * math.log(par["factor"]))
    if kind == "bands":
        turns = par["original"] * f / (2 * math.pi)
        w = ((turns - 1.0) / 3.0).clamp(0.0, 1.0)
        return f * w + f / par["factor"] * (1.0 - w), 1.0
    return f, 1.0


def _rotary(s):
    angle = s["pos"].double()[..., None, None] * s["frequency"]
    cos = (torch.cos(angle) * s["amplitude"]).float()
    sin = (torch.sin(angle) * s["amplitude"]).float()
    rot = s["rot"]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
        if s["layout"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1)
            y = y.flatten(-2)
        return torch.cat([y, x[..., rot:]], -1)

    dtype, page = s["q"].dtype, s["page"]
    q = turned(s["q"], s["q_weight"]).to(dtype)
    s["out"].copy_(torch.where(s["pos"][..., None, None] >= 0, q, s["out"]))
    slot = s["slot"].reshape(-1)
    # rows without a slot write what is there to the last place of the cache,
    # which no row has
    last = s["k_cache"].shape[0] * page - 1
    on = (slot >= 0)[:, None, None]
    at = torch.where(slot >= 0, slot, last)
    for x, cache in ((turned(s["k"], s["k_weight"]).to(dtype), s["k_cache"]),
                     (s["v"], s["v_cache"])):
        x = x.reshape(-1, s["Hkv"], s["D"])
        cache[at // page, :, at % page] = torch.where(
            on, x, cache[-1, :, -1])
    return s["out"], s["k_cache"], s["v_cache"]


def _share(s):
    """Each request picks the page of its context with the most positions
    that others need not read again; requests of one pick share."""
    ctx, n, table = s["ctx"].long(), s["n"].long(), s["table"].long()
    page, P, W, batch = s["page"], s["n_pages"], s["width"], s["batch"]
    dev = table.device
    j = torch.arange(W, device=dev)[None]
    full = torch.where(n >= 0, ctx.clamp(max=W * page - 1) // page, 0)
    known = (j < full[:, None]) & (table >= 0) & (table < P)
    at = torch.where(known, table, P)
    count = torch.zeros(P + 1, dtype=torch.int64, device=dev)
    count.index_add_(0, at.reshape(-1), torch.ones_like(at).reshape(-1))
    gain = torch.where(known, (j + 1) * (count[at] - 1), 0)
    best, d = (gain * W + (W - 1 - j)).max(1)
    most = best // W
    picked = most * page >= s["least"]
    pick = torch.where(picked, at.gather(1, d[:, None])[:, 0], P)
    b = torch.arange(batch, device=dev)
    lead = torch.full((P + 1,), batch, dtype=torch.int64, device=dev)
    lead.scatter_reduce_(0, pick, b, "amin")
    lead = torch.where(picked, lead[pick], b)
    same = ((table == table[lead]) | (j > d[:, None])).all(1)
    member = picked & same & (d == d[lead])
    size = torch.zeros(batch, dtype=torch.int64, device=dev)
    size.index_add_(0, lead, member.long())
    member &= size[lead] > 1
    return (torch.where(member, lead, b).int(),
            torch.where(member, (d + 1) * page, 0).int())


def _attend(s):
    batch, R, Hq, Hkv, D = s["batch"], s["N"] + 1, s["Hq"], s["Hkv"], s["D"]
    G, T, N = Hq // Hkv, s["width"] * s["page"], s["N"]
    at = s["table"].clamp(min=0).long()
    dev = at.device

    def rows(cache):  # [batch][Hkv][T][D]
        return cache[at].permute(0, 2, 1, 3, 4).reshape(
            batch, Hkv, T, D).float()

    ctx, n = s["ctx"].long(), s["n"].long()
    tree = torch.ones(batch, R, R, dtype=torch.bool, device=dev).tril()
    if s["mask"] is not None:
        words = (s["mask"][..., None] >> torch.arange(64, device=dev)) & 1
        tree[:, 1:, 1:] = words.reshape(batch, N, -1)[..., :N] != 0
    r = torch.arange(T, device=dev)[None] - ctx[:, None]
    live = r <= n[:, None]
    seen = tree.gather(2, r.clamp(0, R - 1)[:, None].expand(batch, R, T))
    seen = (r < 0)[:, None] | ((r >= 0) & live)[:, None] & seen
    q = s["q"].reshape(batch, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(
        batch, Hkv, R * G, D).float()
    z = torch.matmul(q, rows(s["k_cache"]).transpose(2, 3)) * s["scale"]
    z = z.view(batch, Hkv, R, G, T).masked_fill_(
        ~seen[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = rows(s["v_cache"]).masked_fill_(~live[:, None, :, None], 0.0)
    out = torch.matmul(p.view(batch, Hkv, R * G, T), v)
    out = out.view(batch, Hkv, R, G, D) / total
    out = out.permute(0, 2, 1, 3, 4).reshape(batch, R, Hq, D)
    lse = (top + total.log()).view(batch, Hkv, R, G).permute(
        0, 2, 1, 3).reshape(batch, R, Hq)
    on = torch.arange(R, device=dev)[None] <= n[:, None]
    out = out.masked_fill(~on[..., None, None], 0.0).to(s["q"].dtype)
    return out, lse.masked_fill(~on[..., None], 0.0)


def _ranked(flags):
    """Place of each set flag among the set ones."""
    return flags.long().cumsum(0) - flags.long()


def _fork(s):
    """The places of dst are emptied, then each becomes a copy of its src's
    context: whole pages shared, the rest copied to a page of its own."""
    batch, W, P, page = s["batch"], s["width"], s["n_pages"], s["page"]
    table, held, ring = s["table"], s["held"], s["ring"]
    dev = table.device
    src, dst = s["src"].long(), s["dst"].long()
    head, count = s["ring_state"].long()
    # pages whose last holder is emptied go to the ring's tail
    ended = torch.zeros(batch + 1, dtype=torch.bool, device=dev)
    ended[torch.where(dst >= 0, dst, batch)] = True
    ended = ended[:batch]
    j = torch.arange(W, device=dev)[None]
    given = ended[:, None] & (j < held.long()[:, None])
    less = torch.zeros(P + 1, dtype=torch.int32, device=dev)
    less.index_add_(0, torch.where(given, table.long(), P).reshape(-1),
                    torch.ones(batch * W, dtype=torch.int32, device=dev))
    extra = s["extra"] - less[:P]
    freed = extra < 0
    extra = extra.clamp(min=0)
    grown = torch.cat([ring, ring[:1]])
    grown[torch.where(freed, (head + count + _ranked(freed)) % P, P)] = \
        torch.arange(P, dtype=torch.int32, device=dev)
    ring.copy_(grown[:P])
    table.copy_(torch.where(given, -1, table))
    ctx = torch.where(ended, 0, s["ctx"].long())
    held_new = torch.where(ended, 0, held.long())
    count = count + freed.sum()
    # forks
    on = (src >= 0) & (dst >= 0)
    a, b = torch.where(on, src, 0), torch.where(on, dst, batch)
    length = torch.where(on, ctx[a], 0)
    full, rest = length // page, length % page
    wants = on & (rest > 0)
    rank = _ranked(wants)
    fits = on & (~wants | (rank < count))
    own_page = ring[(head + rank) % P].long()
    row = torch.where(j < full[:, None], table[a].long(), -1)
    row = torch.where((j == full[:, None]) & wants[:, None],
                      own_page[:, None], row)
    grown = torch.cat([table, table[:1]])
    to = torch.where(fits, b, batch)
    grown[to] = row.int()
    table.copy_(grown[:batch])
    more = torch.cat([extra, extra[:1]])
    shared = fits[:, None] & (j < full[:, None])
    more.index_add_(0, torch.where(shared, row, P).reshape(-1),
                    torch.ones(row.numel(), dtype=torch.int32, device=dev))
    s["extra"].copy_(more[:P])
    for x, y, to_ in ((ctx, length, s["ctx"]),
                      (held_new, full + wants.long(), held)):
        grown = torch.cat([x, x[:1]])
        grown[to] = y
        to_.copy_(grown[:batch])
    taken = (wants & fits).sum()
    s["ring_state"].copy_(torch.stack([(head + taken) % P, count - taken]))
    # forks without a page of their own copy page 0 onto itself
    copied = wants & fits
    from_page = torch.where(copied, table[a].long().gather(
        1, full.clamp(max=W - 1)[:, None])[:, 0], 0)
    to_page = torch.where(copied, own_page, 0)
    keep = (torch.arange(page, device=dev)[None] < torch.where(
        copied, rest, 0)[:, None])[None, :, None, :, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, to_page] = torch.where(keep, cache[:, from_page],
                                        cache[:, to_page])
    return (fits.int(), s["ctx"], table, held, ring, s["ring_state"],
            s["extra"], s["k_cache"], s["v_cache"])


def _compact(s):
    """Pages in use move, in ascending order, to the free ones among the
    first, in ascending order; the ring holds the rest."""
    table, P, W = s["table"].long(), s["n_pages"], s["width"]
    dev = table.device
    mine = torch.arange(W, device=dev)[None] < s["held"].long()[:, None]
    holders = torch.zeros(P + 1, dtype=torch.int64, device=dev)
    at = torch.where(mine, table, P)
    holders.index_add_(0, at.reshape(-1), torch.ones_like(at).reshape(-1))
    holders = holders[:P]
    used = holders > 0
    total = used.sum()
    p = torch.arange(P, device=dev)
    hole, high = ~used & (p < total), used & (p >= total)
    # place P: no page
    holes = torch.full((P + 1,), P, dtype=torch.int64, device=dev)
    holes[torch.where(hole, _ranked(hole), P)] = p
    to = torch.where(high, holes[_ranked(high)], p)
    s["table_new"].copy_(torch.where(
        mine, torch.cat([to, to[:1]])[at], table))
    extra = torch.zeros(P + 1, dtype=torch.int64, device=dev)
    extra[torch.where(used, to, P)] = holders - 1
    s["extra"].copy_(extra[:P])
    s["ring"].copy_((total + p) % P)
    s["ring_state"].copy_(torch.stack([total * 0, P - total]))
    # page[i] moves to the i-th hole; other places move page P - 1 onto itself
    frm = torch.full((P + 1,), P - 1, dtype=torch.int64, device=dev)
    frm[torch.where(high, _ranked(high), P)] = p
    frm = frm[:P // 2 + 1]
    dst = torch.where(torch.arange(len(frm), device=dev) < high.sum(),
                      holes[:len(frm)].clamp(max=P - 1), P - 1)
    # (P - 1 itself, if it is moved, is not a destination)
    frm = torch.where(dst == P - 1, P - 1, frm)
    for cache in (s["k_cache"], s["v_cache"]):
        for layer in cache:
            layer[dst] = layer[frm]
    return (s["table_new"], s["ring"], s["ring_state"], s["extra"],
            s["k_cache"], s["v_cache"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(c, seed):
    if c["op"] == "share":
        return None
    return {"rotary": _exact_rotary, "attend": _exact_attend,
            "fork": _exact_fork, "compact": _exact_compact}[c["op"]](c, seed)


def _exact_rotary(c, seed):
    s = prepare(c, seed)
    rot, half, page = c["rot"], c["rot"] // 2, c["page"]
    par = SCALING[c["scaling"]]
    turns, gain = [], 1.0
    for i in range(half):
        f = math.exp(-2.0 * i / rot * math.log(BASE))
        if c["scaling"] == "linear":
            f /= par["factor"]
        elif c["scaling"] == "base":
            f *= par["factor"] ** (-2.0 * i / (rot - 2))
        elif c["scaling"] == "ramp":
            def pair(r):
                return rot / 2 * math.log(
                    par["original"] / (2 * math.pi * r), BASE)
            lo = max(math.floor(pair(32.0)), 0)
            hi = min(math.ceil(pair(1.0)), rot - 1)
            w = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f *= 1.0 - w + w / par["factor"]
            gain = 0.1 * math.log(par["factor"]) + 1.0
        elif c["scaling"] == "bands":
            w = min(max((par["original"] * f / (2 * math.pi) - 1.0) / 3.0,
                        0.0), 1.0)
            f *= w + (1.0 - w) / par["factor"]
        turns.append(f / (2 * math.pi))
    # whole turns are taken off before the angle is formed
    t = s["pos"].double()[..., None] * torch.tensor(
        turns, dtype=torch.float64, device="cuda")
    t = (t - torch.floor(t)) * (2 * math.pi)
    pair = torch.polar(torch.full_like(t, gain), t)[:, :, None]
    i = torch.arange(half, device="cuda")
    one, two = ((i, i + half) if c["layout"] == "half"
                else (2 * i, 2 * i + 1))
    b = torch.nonzero(s["pos"].reshape(-1) >= 0)[:, 0]

    def rotated(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / c["D"]
                               + EPS) * w.double()
        z = torch.complex(x[..., one], x[..., two]) * pair
        x = x.clone()
        x[..., one], x[..., two] = z.real, z.imag
        return x.reshape(-1, *x.shape[2:])

    out = torch.zeros(c["batch"] * (c["N"] + 1), c["Hq"], c["D"],
                      dtype=torch.float64, device="cuda")
    out[b] = rotated(s["q"], s["q_weight"])[b]
    slot = s["slot"].reshape(-1)[b]
    done = [out.view(c["batch"], c["N"] + 1, c["Hq"], c["D"])]
    for x, cache in ((rotated(s["k"], s["k_weight"]), s["k_cache"]),
                     (s["v"].double().reshape(-1, c["Hkv"], c["D"]),
                      s["v_cache"])):
        flat = cache.double().transpose(1, 2).reshape(-1, c["Hkv"], c["D"])
        flat.index_copy_(0, slot, x[b])
        done.append(flat.view(-1, page, c["Hkv"], c["D"]).transpose(
            1, 2).contiguous())
    return tuple(done)


def _exact_attend(c, seed):
    s = prepare(c, seed)
    R, Hq, Hkv, D, page = c["N"] + 1, c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    out = torch.zeros(c["batch"], R, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["batch"], R, Hq, dtype=torch.float64, device="cuda")
    ctx, n, table = (s[x].cpu().numpy() for x in ("ctx", "n", "table"))
    mask = None if s["mask"] is None else s["mask"].cpu().numpy()
    for b in range(c["batch"]):
        if n[b] < 0:
            continue
        m, L = int(n[b]) + 1, int(ctx[b] + n[b] + 1)
        see = np.zeros((m, L), bool)
        see[:, :L - m + 1] = True
        for i in range(1, m):
            if mask is None:
                see[i, L - m + 1:L - m + 1 + i] = True
            else:
                bits = np.unpackbits(mask[b, i - 1].view(np.uint8),
                                     bitorder="little")
                see[i, L - m + 1:] = bits[:m - 1].astype(bool)
        hidden = torch.from_numpy(~see).cuda()
        pages = torch.from_numpy(
            table[b, :-(-L // page)].astype(np.int64)).cuda()
        k, v = (s[x][pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :L]
                for x in ("k_cache", "v_cache"))
        for h in range(Hkv):
            x = s["q"][b, :m, h * G:(h + 1) * G].double().reshape(m * G, D)
            z = (x @ k[h].double().T).view(m, G, L) * s["scale"]
            z.masked_fill_(hidden[:, None], -math.inf)
            w = torch.softmax(z, -1)
            out[b, :m, h * G:(h + 1) * G] = (
                w.view(m * G, L) @ v[h].double()).view(m, G, D)
            lse[b, :m, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
    return out, lse


def _exact_fork(c, seed):
    s = prepare(c, seed)
    page = c["page"]
    ctx, held, table, extra, ring, state, src, dst = (
        s[x].cpu().numpy().copy() for x in (
            "ctx", "held", "table", "extra", "ring", "ring_state", "src",
            "dst"))
    head, count = int(state[0]), int(state[1])
    back = []
    for b in dst[dst >= 0]:
        for p in table[b, :held[b]]:
            if extra[p] == 0:
                back.append(int(p))
            else:
                extra[p] -= 1
    for p in sorted(back):
        ring[(head + count) % s["n_pages"]] = p
        count += 1
    for a, b in zip(src, dst):
        rest = int(ctx[a]) % page
        if a < 0 or rest == 0:
            continue
        old, new = int(table[a, ctx[a] // page]), int(ring[head])
        head = (head + 1) % s["n_pages"]
        for cache in (s["k_cache"], s["v_cache"]):
            cache[:, new, :, :rest] = cache[:, old, :, :rest]
    return (None,) * 7 + (s["k_cache"].double(), s["v_cache"].double())


def _exact_compact(c, seed):
    s = prepare(c, seed)
    table, held = s["table"].cpu().numpy(), s["held"].cpu().numpy()
    used = sorted({int(p) for b in range(c["batch"])
                   for p in table[b, :held[b]]})
    total = len(used)
    holes = sorted(set(range(total)) - set(used))
    high = [p for p in used if p >= total]
    for a, b in zip(high, holes):
        for cache in (s["k_cache"], s["v_cache"]):
            cache[:, b] = cache[:, a]
    return (None,) * 4 + (s["k_cache"].double(), s["v_cache"].double())
