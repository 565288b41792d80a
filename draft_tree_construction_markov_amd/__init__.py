"""libpctree: draft-tree construction and checking on MI355X (gfx950).

A thin ctypes binding over the C-ABI declared in include/pctree.h.  It only
marshals arguments: torch provides device memory and the current stream;
every step of the computation runs in the library's HIP kernels.  If the
built library is missing the import of any entry point fails loudly: there
is no CPU fallback.

Build it with ``python -m draft_tree_construction_markov_amd.build``.
"""
from __future__ import annotations

import ctypes as C
import functools
import math
import os
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpctree.so")

PCT_F32, PCT_BF16, PCT_F16 = 0, 1, 2
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration",
           3: "workspace too small", 4: "HIP error"}


class PCTError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libpctree: {_STATUS.get(status, status)}: {msg}")
        self.status = status


class TreeShape(C.Structure):
    _fields_ = [("batch", C.c_int32), ("B", C.c_int32), ("V", C.c_int32),
                ("r", C.c_int32), ("k", C.c_int32), ("beam_w", C.c_int32),
                ("N", C.c_int32), ("uw_dtype", C.c_int32)]


class CostModel(C.Structure):
    _fields_ = [("C_d", C.c_double), ("c0", C.c_double), ("c1", C.c_double),
                ("c2", C.c_double), ("c_ell", C.c_double)]


class CacheShape(C.Structure):
    _fields_ = [("batch", C.c_int32), ("N", C.c_int32),
                ("n_pages", C.c_int32), ("page_size", C.c_int32),
                ("max_pages", C.c_int32), ("Hq", C.c_int32),
                ("Hkv", C.c_int32), ("D", C.c_int32), ("dtype", C.c_int32)]


class RotaryDesc(C.Structure):
    _fields_ = [("rot", C.c_int32), ("layout", C.c_int32),
                ("scaling", C.c_int32), ("original", C.c_int32),
                ("base", C.c_double), ("factor", C.c_double),
                ("low", C.c_double), ("high", C.c_double),
                ("amplitude", C.c_double)]


class _PageState(C.Structure):
    _fields_ = [(x, C.c_void_p) for x in (
        "ctx_len", "block_table", "n_held", "ring", "ring_state", "extra")]


_lib = None


def lib():
    """Load libpctree.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FileNotFoundError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m draft_tree_construction_markov_amd.build`")
    L = C.CDLL(LIB_PATH)
    P, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    L.pct_markov_logits.argtypes = [P, i64, i32, P, P, i32, i32, i32, P, P,
                                    i32, i32, P, P, P, P, P, sz, P]
    L.pct_markov_logits_workspace.argtypes = [i32, i32, i32]
    L.pct_markov_logits_workspace.restype = sz
    L.pct_build_tree.argtypes = [C.POINTER(TreeShape), P, P, P, P, P, P, P, P,
                                 P, P, P, sz, P]
    L.pct_build_tree_workspace.argtypes = [C.POINTER(TreeShape)]
    L.pct_build_tree_workspace.restype = sz
    L.pct_tree_mask.argtypes = [i32, i32, P, P, P, P]
    L.pct_verify_accept.argtypes = [i32, i32, i32, P, P, P, P, P, P, P, P, P,
                                    P]
    if hasattr(L, "pct_build_tree_adaptive"):
        L.pct_build_tree_adaptive.argtypes = [
            i32, i32, i32, i32, P, P, C.POINTER(CostModel), P, P, P, P, P, P,
            P, P, P, sz, P]
        L.pct_build_tree_adaptive_workspace.argtypes = [i32, i32, i32, i32]
        L.pct_build_tree_adaptive_workspace.restype = sz
    L.pct_build_tree_adaptive_pc.argtypes = [
        C.POINTER(TreeShape), P, P, P, P, P, C.POINTER(CostModel), P, P, P, P,
        P, P, P, P, P, sz, P]
    L.pct_build_tree_adaptive_pc_workspace.argtypes = [C.POINTER(TreeShape)]
    L.pct_build_tree_adaptive_pc_workspace.restype = sz
    L.pct_throughput_curve.argtypes = [i32, i32, P, P, P,
                                       C.POINTER(CostModel), P, P]
    L.pct_verify_sample.argtypes = [i32, i32, i32, i32, P, P, P, P, P, P,
                                    C.c_double, C.c_uint64, P, P, P, P, P,
                                    sz, P]
    L.pct_verify_sample_workspace.argtypes = [i32, i32, i32]
    L.pct_verify_sample_workspace.restype = sz
    shape = C.POINTER(CacheShape)
    L.pct_cache_plan_workspace.argtypes = [i32]
    L.pct_cache_plan_workspace.restype = sz
    L.pct_cache_plan.argtypes = [shape, P, P, P, P, P, P, P, P, P, P, P, sz,
                                 P]
    L.pct_cache_plan_served.argtypes = [shape, P, P, P, P, P, P, P, P, P, P,
                                        P, P, sz, P]
    L.pct_cache_write.argtypes = [shape, P, i64, P, i64, P, P, P, P]
    L.pct_rotary_table.argtypes = [C.POINTER(RotaryDesc), P]
    L.pct_cache_write_rotary.argtypes = [
        shape, C.POINTER(RotaryDesc), P, C.c_float, P, P, P, i64, P, i64, P,
        i64, P, P, P, i64, P, P, P]
    state = C.POINTER(_PageState)
    for name in ("free", "compact"):
        f = getattr(L, f"pct_cache_{name}_workspace")
        f.argtypes, f.restype = [shape], sz
    L.pct_cache_fork_workspace.argtypes = [shape, i32]
    L.pct_cache_fork_workspace.restype = sz
    L.pct_cache_free.argtypes = [shape, i32, P, state, P, sz, P]
    L.pct_cache_trim.argtypes = [shape, P, state, P, sz, P]
    L.pct_cache_fork.argtypes = [shape, i32, i64, i32, P, P, P, state, P, P,
                                 P, P, sz, P]
    L.pct_cache_compact.argtypes = [shape, i32, i64, state, P, P, P, P, sz, P]
    for name in ("cache_share_size", "cache_share_workspace",
                 "shared_attention_workspace"):
        f = getattr(L, f"pct_{name}")
        f.argtypes, f.restype = [shape], sz
    L.pct_cache_share.argtypes = [shape, i32, P, P, P, P, P, P, P, sz, P]
    L.pct_shared_attention.argtypes = [shape, C.c_float, P, i64, P, P, P, P,
                                       P, P, P, P, sz, P]
    L.pct_tree_attention_workspace.argtypes = [shape]
    L.pct_tree_attention_workspace.restype = sz
    L.pct_tree_attention.argtypes = [shape, C.c_float, P, i64, P, P, P, P, P,
                                     P, P, P, P, sz, P]
    L.pct_cache_commit.argtypes = [shape, i32, i64, i32, P, P, P, P, P, P, P,
                                   P, P]
    L.pct_profile_enable.argtypes = [i32]
    L.pct_profile_reset.argtypes = []
    L.pct_profile_read.argtypes = [i32, i64, C.POINTER(C.c_double),
                                   C.POINTER(C.c_int64)]
    L.pct_last_error.restype = C.c_char_p
    L.pct_status_string.restype = C.c_char_p
    _lib = L
    return L


def exported_symbols():
    """Names of the C-ABI entry points the header declares."""
    return ["pct_markov_logits", "pct_markov_logits_workspace",
            "pct_build_tree", "pct_build_tree_workspace",
            "pct_build_tree_adaptive", "pct_build_tree_adaptive_workspace",
            "pct_build_tree_adaptive_pc",
            "pct_build_tree_adaptive_pc_workspace", "pct_throughput_curve",
            "pct_build_tree_noalloc", "pct_verify_sample",
            "pct_verify_sample_workspace",
            "pct_tree_mask", "pct_verify_accept",
            "pct_cache_plan", "pct_cache_plan_served",
            "pct_cache_plan_workspace", "pct_cache_write",
            "pct_rotary_table", "pct_cache_write_rotary",
            "pct_cache_free", "pct_cache_trim", "pct_cache_free_workspace",
            "pct_cache_fork", "pct_cache_fork_workspace",
            "pct_cache_compact", "pct_cache_compact_workspace",
            "pct_cache_share", "pct_cache_share_size",
            "pct_cache_share_workspace", "pct_shared_attention",
            "pct_shared_attention_workspace",
            "pct_tree_attention", "pct_tree_attention_workspace",
            "pct_cache_commit", "pct_profile_enable",
            "pct_profile_reset", "pct_profile_read", "pct_status_string",
            "pct_last_error"]


PROF_MARKOV, PROF_EXPAND, PROF_TOPN, PROF_MASK, PROF_ACCEPT, PROF_ROWTOP, \
    PROF_INIT, PROF_ROWSTATS, PROF_BESTFIRST, PROF_FINALIZE, PROF_STOP, \
    PROF_SAMPLE, PROF_PLAN, PROF_CACHE_WRITE, PROF_ATTEND, PROF_JOIN, \
    PROF_COMMIT, PROF_ROTARY, PROF_RELEASE, PROF_FORK, \
    PROF_COMPACT, PROF_SHARE = range(22)


def profile_enable(on: bool = True):
    _check(lib().pct_profile_enable(1 if on else 0))


def profile_reset():
    _check(lib().pct_profile_reset())


def profile_read(kind: int, units: int = -1):
    """(total milliseconds, launches) recorded for one kernel kind."""
    ms = C.c_double()
    n = C.c_int64()
    _check(lib().pct_profile_read(kind, units, C.byref(ms), C.byref(n)))
    return ms.value, n.value


def _check(rc: int):
    if rc != 0:
        raise PCTError(rc, lib().pct_last_error().decode())


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(device) -> C.c_void_p:
    return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dev(t: torch.Tensor):
    if not t.is_cuda:
        raise ValueError("libpctree needs device tensors")
    return t.device


def _factors(U, W):
    if U is None and W is None:
        return None, None, PCT_F32, 0
    if U is None or W is None:
        raise ValueError("U and W must both be given or both None")
    if U.dtype != W.dtype or U.shape != W.shape or U.dim() != 2:
        raise ValueError("U and W must be [V][r] tensors of the same dtype")
    if U.dtype == torch.bfloat16:
        dt = PCT_BF16
    elif U.dtype == torch.float32:
        dt = PCT_F32
    else:
        raise ValueError("U/W must be bfloat16 or float32")
    return U.contiguous(), W.contiguous(), dt, int(U.shape[1])


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# pct_markov_logits

def markov_logits(L, U, W, parent_tok, parent_Lrow, k: int,
                  want_z: bool = False, V: int | None = None):
    """Per-parent lse and top-k of z = L[row] + U[tok] . W[v].
    L: [rows][V] float32 or None; U, W: [V][r] or None.
    Returns (lse [P], topk_tok [P][k], topk_logp [P][k], z [P][V] or None)."""
    dev = _dev(parent_tok)
    U, W, dt, r = _factors(U, W)
    if L is not None:
        L = L.contiguous()
        V = int(L.shape[-1])
        stride = V
        rows = int(L.numel() // V)
    else:
        V = int(U.shape[0])
        stride = 0
        rows = 0
    P = int(parent_tok.numel())
    lse = torch.empty(P, dtype=torch.float32, device=dev)
    tt = torch.empty(P, k, dtype=torch.int32, device=dev)
    tl = torch.empty(P, k, dtype=torch.float32, device=dev)
    z = torch.empty(P, V, dtype=torch.float32, device=dev) if want_z else None
    nbytes = lib().pct_markov_logits_workspace(P, V, k)
    ws = _workspace(nbytes, dev)
    pt = parent_tok.to(torch.int32).contiguous()
    pr = None if parent_Lrow is None else parent_Lrow.to(torch.int32).contiguous()
    _check(lib().pct_markov_logits(
        _ptr(L), stride, rows, _ptr(U), _ptr(W), dt, V, r, _ptr(pt), _ptr(pr), P, k,
        _ptr(lse), _ptr(tt), _ptr(tl), _ptr(z), _ptr(ws), ws.numel(),
        _stream(dev)))
    return lse, tt, tl, z


# ---------------------------------------------------------------------------
# pct_build_tree

@dataclass
class TreeOutputs:
    tok: torch.Tensor
    parent: torch.Tensor
    depth: torch.Tensor
    score: torch.Tensor
    n_nodes: torch.Tensor
    mask: torch.Tensor | None

    def numpy(self):
        out = {k: getattr(self, k).cpu().numpy()
               for k in ("tok", "parent", "depth", "score", "n_nodes")}
        if self.mask is not None:
            out["mask"] = self.mask.cpu().numpy().view("uint64")
        return out


class TreeBuilder:
    """A parent-conditioned build of fixed shape with its workspace and
    outputs allocated once; run() only enqueues kernels."""

    def __init__(self, batch: int, B: int, V: int, k: int, beam_w: int,
                 N: int, r: int = 0, bf16: bool = True, mask: bool = False,
                 device="cuda"):
        self.shape = TreeShape(batch, B, V, r, k, beam_w, N,
                               PCT_BF16 if bf16 else PCT_F32)
        self.device = torch.device(device)
        nbytes = lib().pct_build_tree_workspace(C.byref(self.shape))
        if nbytes == 0:
            raise PCTError(1, lib().pct_last_error().decode())
        self.ws = _workspace(nbytes, self.device)
        dev = self.device
        words = (N + 63) // 64
        self.out = TreeOutputs(
            tok=torch.empty(batch, N, dtype=torch.int32, device=dev),
            parent=torch.empty(batch, N, dtype=torch.int32, device=dev),
            depth=torch.empty(batch, N, dtype=torch.int32, device=dev),
            score=torch.empty(batch, N, dtype=torch.float32, device=dev),
            n_nodes=torch.empty(batch, dtype=torch.int32, device=dev),
            mask=(torch.empty(batch, N, words, dtype=torch.int64, device=dev)
                  if mask else None))

    def run(self, L, U, W, anchor) -> TreeOutputs:
        o = self.out
        _check(lib().pct_build_tree(
            C.byref(self.shape), _ptr(L), _ptr(U), _ptr(W), _ptr(anchor),
            _ptr(o.tok), _ptr(o.parent), _ptr(o.depth), _ptr(o.score),
            _ptr(o.n_nodes), _ptr(o.mask), _ptr(self.ws), self.ws.numel(),
            _stream(self.device)))
        return o


def build_tree(L, U, W, anchor, k: int, beam_w: int, N: int,
               mask: bool = False) -> TreeOutputs:
    """PCTree on L [batch][B][V] float32 with factors U, W [V][r] (bf16 or
    fp32) or None; anchor [batch] int32."""
    dev = _dev(L)
    batch, B, V = (int(x) for x in L.shape)
    U, W, dt, r = _factors(U, W)
    tb = TreeBuilder(batch, B, V, k, beam_w, N, r=r, bf16=(dt == PCT_BF16),
                     mask=mask, device=dev)
    return tb.run(L.contiguous(), U, W, anchor.to(torch.int32).contiguous())


# ---------------------------------------------------------------------------
# pct_build_tree_adaptive

class AdaptiveBuilder:
    """CaDDTree best-first build with the throughput stop, fixed shape."""

    def __init__(self, batch: int, B: int, V: int, n_max: int,
                 cost: dict | None, mask: bool = False, device="cuda"):
        self.batch, self.B, self.V, self.n_max = batch, B, V, n_max
        self.cost = None if cost is None else CostModel(
            cost["C_d"], cost["c0"], cost["c1"], cost["c2"], cost["c_ell"])
        self.device = torch.device(device)
        nbytes = lib().pct_build_tree_adaptive_workspace(batch, B, V, n_max)
        if nbytes == 0:
            raise PCTError(1, lib().pct_last_error().decode())
        self.ws = _workspace(nbytes, self.device)
        dev = self.device
        words = (n_max + 63) // 64
        self.tok = torch.empty(batch, n_max, dtype=torch.int32, device=dev)
        self.parent = torch.empty_like(self.tok)
        self.depth = torch.empty_like(self.tok)
        self.score = torch.empty(batch, n_max, dtype=torch.float32, device=dev)
        self.n_star = torch.empty(batch, dtype=torch.int32, device=dev)
        self.phi = torch.empty(batch, dtype=torch.float64, device=dev)
        self.throughput = torch.empty(batch, dtype=torch.float64, device=dev)
        self.mask = (torch.empty(batch, n_max, words, dtype=torch.int64,
                                 device=dev) if mask else None)

    def run(self, L, ctx_len):
        _check(lib().pct_build_tree_adaptive(
            self.batch, self.B, self.V, self.n_max, _ptr(L), _ptr(ctx_len),
            None if self.cost is None else C.byref(self.cost),
            _ptr(self.tok), _ptr(self.parent), _ptr(self.depth),
            _ptr(self.score), _ptr(self.n_star), _ptr(self.phi),
            _ptr(self.throughput), _ptr(self.mask), _ptr(self.ws),
            self.ws.numel(), _stream(self.device)))
        return self

    def numpy(self):
        out = {k: getattr(self, k).cpu().numpy()
               for k in ("tok", "parent", "depth", "score", "n_star", "phi",
                         "throughput")}
        if self.mask is not None:
            out["mask"] = self.mask.cpu().numpy().view("uint64")
        return out


def build_tree_adaptive(L, ctx_len, n_max: int, cost: dict | None,
                        mask: bool = False) -> AdaptiveBuilder:
    batch, B, V = (int(x) for x in L.shape)
    ab = AdaptiveBuilder(batch, B, V, n_max, cost, mask=mask,
                         device=_dev(L))
    return ab.run(L.contiguous(), ctx_len.to(torch.int32).contiguous())


# ---------------------------------------------------------------------------
# pct_build_tree_adaptive_pc / pct_throughput_curve

def _cost_struct(cost):
    return None if cost is None else CostModel(
        cost["C_d"], cost["c0"], cost["c1"], cost["c2"], cost["c_ell"])


class AdaptivePCBuilder:
    """Throughput stop on the parent-conditioned tree, fixed shape (N is
    the largest tree considered)."""

    def __init__(self, batch: int, B: int, V: int, k: int, beam_w: int,
                 n_max: int, cost: dict | None, r: int = 0,
                 bf16: bool = True, mask: bool = False, device="cuda"):
        self.shape = TreeShape(batch, B, V, r, k, beam_w, n_max,
                               PCT_BF16 if bf16 else PCT_F32)
        self.cost = _cost_struct(cost)
        self.device = torch.device(device)
        nbytes = lib().pct_build_tree_adaptive_pc_workspace(
            C.byref(self.shape))
        if nbytes == 0:
            raise PCTError(1, lib().pct_last_error().decode())
        self.ws = _workspace(nbytes, self.device)
        dev = self.device
        words = (n_max + 63) // 64
        self.tok = torch.empty(batch, n_max, dtype=torch.int32, device=dev)
        self.parent = torch.empty_like(self.tok)
        self.depth = torch.empty_like(self.tok)
        self.score = torch.empty(batch, n_max, dtype=torch.float32, device=dev)
        self.n_star = torch.empty(batch, dtype=torch.int32, device=dev)
        self.phi = torch.empty(batch, dtype=torch.float64, device=dev)
        self.throughput = torch.empty(batch, dtype=torch.float64, device=dev)
        self.mask = (torch.empty(batch, n_max, words, dtype=torch.int64,
                                 device=dev) if mask else None)

    def run(self, L, U, W, anchor, ctx_len):
        _check(lib().pct_build_tree_adaptive_pc(
            C.byref(self.shape), _ptr(L), _ptr(U), _ptr(W), _ptr(anchor),
            _ptr(ctx_len), None if self.cost is None else C.byref(self.cost),
            _ptr(self.tok), _ptr(self.parent), _ptr(self.depth),
            _ptr(self.score), _ptr(self.n_star), _ptr(self.phi),
            _ptr(self.throughput), _ptr(self.mask), _ptr(self.ws),
            self.ws.numel(), _stream(self.device)))
        return self

    def numpy(self):
        out = {k: getattr(self, k).cpu().numpy()
               for k in ("tok", "parent", "depth", "score", "n_star", "phi",
                         "throughput")}
        if self.mask is not None:
            out["mask"] = self.mask.cpu().numpy().view("uint64")
        return out


def build_tree_adaptive_pc(L, U, W, anchor, ctx_len, k: int, beam_w: int,
                           n_max: int, cost: dict | None,
                           mask: bool = False) -> AdaptivePCBuilder:
    dev = _dev(L)
    batch, B, V = (int(x) for x in L.shape)
    U, W, dt, r = _factors(U, W)
    ab = AdaptivePCBuilder(batch, B, V, k, beam_w, n_max, cost, r=r,
                           bf16=(dt == PCT_BF16), mask=mask, device=dev)
    return ab.run(L.contiguous(), U, W, anchor.to(torch.int32).contiguous(),
                  ctx_len.to(torch.int32).contiguous())


def throughput_curve(score, n_nodes, ctx_len, cost: dict | None):
    """f(n) = (1 + Phi_n) / D(n) for n = 0..N of best-first-ordered scores
    [batch][N]; returns [batch][N+1] float64."""
    dev = _dev(score)
    batch, N = (int(x) for x in score.shape)
    f = torch.empty(batch, N + 1, dtype=torch.float64, device=dev)
    cm = _cost_struct(cost)
    _check(lib().pct_throughput_curve(
        batch, N, _ptr(score.contiguous()), _ptr(n_nodes.contiguous()),
        _ptr(None if ctx_len is None else ctx_len.contiguous()),
        None if cm is None else C.byref(cm), _ptr(f), _stream(dev)))
    return f


# ---------------------------------------------------------------------------
# pct_tree_mask / pct_verify_accept

def tree_mask(parent, n_nodes, out=None) -> torch.Tensor:
    """parent [batch][N] int32, n_nodes [batch] -> mask [batch][N][words]
    (int64 storage of the uint64 words), into `out` when given."""
    dev = _dev(parent)
    batch, N = (int(x) for x in parent.shape)
    words = (N + 63) // 64
    mask = out if out is not None else torch.empty(
        batch, N, words, dtype=torch.int64, device=dev)
    if tuple(mask.shape) != (batch, N, words) or mask.dtype != torch.int64:
        raise ValueError("mask must be int64 [batch][N][ceil(N/64)]")
    _check(lib().pct_tree_mask(batch, N, _ptr(parent.contiguous()),
                               _ptr(n_nodes.contiguous()), _ptr(mask),
                               _stream(dev)))
    return mask


def verify_accept(tok, parent, depth, n_nodes, target, B: int, out=None,
                  mask=None):
    """Greedy acceptance walk; with the tree's packed ancestry mask the
    acceptance test uses it.  Returns (tau [batch], accept_node [batch][B],
    accept_tok [batch][B+1])."""
    dev = _dev(tok)
    batch, N = (int(x) for x in tok.shape)
    if out is None:
        out = (torch.empty(batch, dtype=torch.int32, device=dev),
               torch.empty(batch, B, dtype=torch.int32, device=dev),
               torch.empty(batch, B + 1, dtype=torch.int32, device=dev))
    if mask is not None and tuple(mask.shape) != (batch, N, (N + 63) // 64):
        raise ValueError("mask must be [batch][N][ceil(N/64)]")
    tau, an, at = out
    _check(lib().pct_verify_accept(
        batch, N, B, _ptr(tok), _ptr(parent), _ptr(depth), _ptr(n_nodes),
        _ptr(mask), _ptr(target), _ptr(tau), _ptr(an), _ptr(at),
        _stream(dev)))
    return tau, an, at


def verify_sample(tok, parent, depth, n_nodes, target_logits, B: int,
                  temperature: float, seed: int, mask=None, out=None,
                  workspace=None):
    """Verification with temperature sampling: target_logits
    [batch][N+1][V] float32.  Returns (sampled [batch][N+1], tau [batch],
    accept_node [batch][B], accept_tok [batch][B+1]).  workspace: an
    optional uint8 device tensor reused across calls."""
    dev = _dev(tok)
    batch, N = (int(x) for x in tok.shape)
    V = int(target_logits.shape[-1])
    if tuple(target_logits.shape) != (batch, N + 1, V):
        raise ValueError("target_logits must be [batch][N+1][V]")
    if out is None:
        out = (torch.empty(batch, N + 1, dtype=torch.int32, device=dev),
               torch.empty(batch, dtype=torch.int32, device=dev),
               torch.empty(batch, B, dtype=torch.int32, device=dev),
               torch.empty(batch, B + 1, dtype=torch.int32, device=dev))
    sm, tau, an, at = out
    nb = int(lib().pct_verify_sample_workspace(batch, N, V))
    if workspace is None or workspace.numel() < nb:
        workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
    _check(lib().pct_verify_sample(
        batch, N, B, V, _ptr(tok), _ptr(parent), _ptr(depth), _ptr(n_nodes),
        _ptr(mask), _ptr(target_logits.contiguous()), float(temperature),
        int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(sm), _ptr(tau), _ptr(an),
        _ptr(at), _ptr(workspace), workspace.numel(), _stream(dev)))
    return sm, tau, an, at


# ---------------------------------------------------------------------------
# paged key-value cache: pct_cache_plan / pct_cache_write /
# pct_tree_attention / pct_cache_commit

_CACHE_TYPES = {torch.bfloat16: PCT_BF16, torch.float16: PCT_F16}


def _cache_dtype(dtype) -> int:
    if dtype not in _CACHE_TYPES:
        raise ValueError("the cache holds bfloat16 or float16")
    return _CACHE_TYPES[dtype]


def _want(name, t, dtype, shape, dev):
    """Check one tensor of a cache call (dev: device index) and return its
    address."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev and
            t.is_contiguous()):
        return t.data_ptr()
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on device {dev}")
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape "
                     f"{tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


@functools.lru_cache(maxsize=64)
def _shape_ref(*fields):
    """A reference to the shape structure of these fields (read only)."""
    return C.byref(CacheShape(*fields))


def _rows(name, t, dtype, shape, dev):
    """Check rows [batch][R][heads][D] whose heads are contiguous and whose
    rows are evenly spaced (a joint projection's view); returns the address
    and the row stride."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} tensor of shape "
                         f"{tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on device {dev}")
    b, R, H, D = shape
    sb, sr, sh, sd = t.stride()
    if R == 1:
        sr = sb if b > 1 else H * D
    if ((sd != 1 and D > 1) or (sh != D and H > 1) or
            (b > 1 and sb != R * sr)):
        raise ValueError(f"{name} needs contiguous heads and evenly spaced "
                         f"rows, got strides {t.stride()}")
    return t.data_ptr(), sr


def _enqueue(fn, dev: int, *args):
    """Call a cache entry point on the current stream of device `dev`, which
    is made current for the call when it is not."""
    cuda = torch._C
    if cuda._cuda_getDevice() == dev:
        rc = fn(*args, cuda._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, cuda._cuda_getCurrentRawStream(dev))
    if rc != 0:
        _check(rc)


def _device(device) -> torch.device:
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


@dataclass
class CacheRows:
    """Where a round's rows go: slot [batch][N+1] int64 (-1: none), pos
    [batch][N+1] int32 (place in the sequence, -1 for unused rows), missing
    [batch] int32 (pages that the free ring could not give), n_served [batch]
    int32 (n_nodes, -1 for the requests that miss pages: the n_nodes of the
    round's attention and commit)."""
    slot: torch.Tensor
    pos: torch.Tensor
    missing: torch.Tensor
    n_served: torch.Tensor | None = None


class CachePlan:
    """Page plan of fixed shape with its workspace and outputs allocated
    once; run() only enqueues kernels."""

    def __init__(self, batch: int, N: int, n_pages: int, page_size: int,
                 max_pages: int, device="cuda"):
        self.shape = CacheShape(batch, N, n_pages, page_size, max_pages, 1, 1,
                                16, PCT_BF16)
        self.device = dev = _device(device)
        self.ws = _workspace(lib().pct_cache_plan_workspace(batch), dev)
        i32 = dict(dtype=torch.int32, device=dev)
        # no slots and no rows before the first run
        self.out = CacheRows(
            slot=torch.full((batch, N + 1), -1, dtype=torch.int64,
                            device=dev),
            pos=torch.full((batch, N + 1), -1, **i32),
            missing=torch.zeros(batch, **i32),
            n_served=torch.full((batch,), -1, **i32))
        o = self.out
        self._fn, self._ref = lib().pct_cache_plan_served, C.byref(self.shape)
        self._shapes = ((batch,), (batch, N), (batch, max_pages), (n_pages,),
                        (2,))
        self._tail = tuple(C.c_void_p(x.data_ptr()) for x in (
            o.slot, o.pos, o.missing, o.n_served, self.ws)) + (
                self.ws.numel(),)

    def _depth(self, depth):
        nodes = self._shapes[1]
        if nodes[1] == 0:
            return None
        if depth is None:
            raise ValueError("depth is required when N > 0")
        return _want("depth", depth, torch.int32, nodes, self.device.index)

    def run(self, ctx_len, n_nodes, block_table, n_held, ring, ring_state,
            depth=None) -> CacheRows:
        """n_nodes None = N everywhere; depth [batch][N] gives nodes their
        place in the sequence and is required unless N = 0."""
        dev, i32 = self.device.index, torch.int32
        one, _, pages, free, state = self._shapes
        dp = self._depth(depth)
        _enqueue(self._fn, dev, self._ref,
                 _want("ctx_len", ctx_len, i32, one, dev),
                 None if n_nodes is None else
                 _want("n_nodes", n_nodes, i32, one, dev), dp,
                 _want("block_table", block_table, i32, pages, dev),
                 _want("n_held", n_held, i32, one, dev),
                 _want("ring", ring, i32, free, dev),
                 _want("ring_state", ring_state, i32, state, dev),
                 *self._tail)
        return self.out


def cache_write(k, v, slot, k_cache, v_cache):
    """Write the rows k, v [batch][R][Hkv][D] (views with evenly spaced rows
    allowed) into slots slot [batch][R] of k_cache, v_cache
    [n_pages][Hkv][page_size][D]; a slot outside the cache is left out."""
    dev = k_cache.get_device()
    if dev < 0:
        raise ValueError("libpctree needs device tensors")
    cache = k_cache.shape
    n_pages, Hkv, page, D = cache
    batch, R = slot.shape
    dt = k_cache.dtype
    rows = (batch, R, Hkv, D)
    sh = _shape_ref(batch, R - 1, n_pages, page, 1, Hkv, Hkv, D,
                    _cache_dtype(dt))
    kp, ks = _rows("k", k, dt, rows, dev)
    vp, vs = _rows("v", v, dt, rows, dev)
    _enqueue(lib().pct_cache_write, dev, sh, kp, ks, vp, vs,
             _want("slot", slot, torch.int64, (batch, R), dev),
             _want("k_cache", k_cache, dt, cache, dev),
             _want("v_cache", v_cache, dt, cache, dev))


class Rotary:
    """Rotary positions of heads of D elements: which are rotated and how
    fast, with the table of frequencies on the device.

    rot: rotated elements, the first of each head (default: all; 0: none).
    layout: "half" (pairs i, i + rot/2) or "interleaved" (2i, 2i + 1).
    Pair i turns by base^(-2i/rot) radians per position, for long contexts
    scaled by `factor`: "linear" (all pairs), "base" (a larger base), "ramp"
    (slow pairs, by a ramp over the pairs between those that make `high` and
    `low` turns over `original` positions; 32 and 1), "bands" (slow pairs, by
    a ramp over their turns; 4 and 1).  amplitude: factor of the rotated
    elements (default 1; 1 + 0.1 ln(factor) for a "ramp" of factor > 1)."""

    LAYOUTS = ("half", "interleaved")
    SCALINGS = ("none", "linear", "base", "ramp", "bands")

    def __init__(self, D: int, rot: int | None = None, base: float = 10000.0,
                 layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, original: int = 0,
                 low: float | None = None, high: float | None = None,
                 amplitude: float | None = None, device="cuda"):
        if layout not in self.LAYOUTS:
            raise ValueError(f"layout must be one of {self.LAYOUTS}")
        if scaling not in self.SCALINGS:
            raise ValueError(f"scaling must be one of {self.SCALINGS}")
        rot = D if rot is None else rot
        if rot > D:
            raise ValueError(f"rot = {rot} exceeds D = {D}")
        if low is None:
            low = 1.0
        if high is None:
            high = 32.0 if scaling == "ramp" else 4.0
        if amplitude is None:
            amplitude = (1.0 + 0.1 * math.log(factor)
                         if scaling == "ramp" and factor > 1.0 else 1.0)
        self.D = D
        self.desc = RotaryDesc(rot, self.LAYOUTS.index(layout),
                               self.SCALINGS.index(scaling), original, base,
                               factor, low, high, amplitude)
        self._ref = C.byref(self.desc)
        table = torch.zeros(max(rot, 0) // 2, dtype=torch.int64)
        _check(lib().pct_rotary_table(self._ref, table.data_ptr()))
        self.table = table.to(_device(device))
        self._dev = self.table.get_device()
        self._table = self.table.data_ptr()


def cache_write_rotary(rotary: Rotary, q, k, v, pos, slot, k_cache, v_cache,
                       q_weight=None, k_weight=None, eps: float = 1e-6,
                       out=None):
    """Queries q [batch][R][Hq][D] and keys k [batch][R][Hkv][D] (views with
    evenly spaced rows allowed), normalised if weights [D] (float32) are
    given, rotated to positions pos [batch][R] int32: keys, with the values
    v as they are, into slots slot [batch][R] of k_cache, v_cache
    [n_pages][Hkv][page_size][D], queries into `out` (may be q itself;
    default: a new tensor of zeros), which is returned.  Rows of negative
    positions are left out, and `out` keeps what it held there.  q, or k and
    v, may be None."""
    dev = k_cache.get_device()
    if dev < 0:
        raise ValueError("libpctree needs device tensors")
    if rotary._dev != dev:
        raise ValueError(f"the rotary table is on {rotary.table.device}, not "
                         f"on device {dev}")
    cache = k_cache.shape
    n_pages, Hkv, page, D = cache
    if D != rotary.D:
        raise ValueError(f"the rotary table is for heads of {rotary.D} "
                         f"elements, the cache has {D}")
    if (k is None) != (v is None) or (q is None and k is None):
        raise ValueError("need q, or k and v, or all of them")
    batch, R = pos.shape
    dt = k_cache.dtype
    kp = vp = qp = op = None
    ks = vs = qs = os_ = 0
    Hq = Hkv
    if q is not None:
        Hq = q.shape[-2]
        rows = (batch, R, Hq, D)
        qp, qs = _rows("q", q, dt, rows, dev)
        if out is None:
            out = torch.zeros(rows, dtype=dt, device=q.device)
        op, os_ = _rows("out", out, dt, rows, dev)
    if k is not None:
        rows = (batch, R, Hkv, D)
        kp, ks = _rows("k", k, dt, rows, dev)
        vp, vs = _rows("v", v, dt, rows, dev)
    f32, wide = torch.float32, (D,)
    _enqueue(lib().pct_cache_write_rotary, dev,
             _shape_ref(batch, R - 1, n_pages, page, 1, Hq, Hkv, D,
                        _cache_dtype(dt)),
             rotary._ref, rotary._table, eps,
             None if q_weight is None else
             _want("q_weight", q_weight, f32, wide, dev),
             None if k_weight is None else
             _want("k_weight", k_weight, f32, wide, dev),
             qp, qs, kp, ks, vp, vs,
             _want("pos", pos, torch.int32, (batch, R), dev),
             None if k is None else
             _want("slot", slot, torch.int64, (batch, R), dev),
             op, os_, _want("k_cache", k_cache, dt, cache, dev),
             _want("v_cache", v_cache, dt, cache, dev))
    return out if q is not None else None


class TreeAttention:
    """Attention of a round's rows over a paged cache, fixed shape, with its
    workspace and outputs allocated once; run() only enqueues kernels.  Its
    outputs carry no gradient."""

    def __init__(self, batch: int, N: int, Hq: int, Hkv: int, D: int,
                 n_pages: int, page_size: int, max_pages: int,
                 dtype=torch.bfloat16, lse: bool = False, device="cuda"):
        self.dtype = dtype
        self.shape = CacheShape(batch, N, n_pages, page_size, max_pages, Hq,
                                Hkv, D, _cache_dtype(dtype))
        self.device = dev = _device(device)
        self._fn, self._ref = lib().pct_tree_attention, C.byref(self.shape)
        nbytes = lib().pct_tree_attention_workspace(self._ref)
        if nbytes == 0:
            raise PCTError(1, lib().pct_last_error().decode())
        self.ws = _workspace(nbytes, dev)
        # a call writes the rows it uses: those that none has used stay zero
        self.out = torch.zeros(batch, N + 1, Hq, D, dtype=dtype, device=dev)
        self.lse = (torch.zeros(batch, N + 1, Hq, dtype=torch.float32,
                                device=dev) if lse else None)
        self._shapes = ((batch, N + 1, Hq, D), (n_pages, Hkv, page_size, D),
                        (batch, max_pages), (batch,),
                        (batch, N, (N + 63) // 64))
        self._op = C.c_void_p(self.out.data_ptr())
        self._tail = (None if self.lse is None else
                      C.c_void_p(self.lse.data_ptr()),
                      C.c_void_p(self.ws.data_ptr()), self.ws.numel())

    def run(self, q, k_cache, v_cache, block_table, ctx_len, n_nodes=None,
            mask=None, scale=None, out=None):
        """q [batch][N+1][Hq][D] (a view with evenly spaced rows allowed),
        mask [batch][N][ceil(N/64)] int64 or None (straight drafts); scale
        defaults to 1/sqrt(D).  Returns (out, lse), lse None unless the
        handle keeps it; out: another tensor for the outputs.

        The handle's tensors are written by every call: clone what is needed
        past the next one.  Rows past n_nodes are left as they were: they
        hold what an earlier call wrote there, or zeros."""
        dev, dt, i32 = self.device.index, self.dtype, torch.int32
        rows, cache, pages, one, words = self._shapes
        if out is None:
            out, op = self.out, self._op
        else:
            op = _want("out", out, dt, rows, dev)
        qp, qs = _rows("q", q, dt, rows, dev)
        _enqueue(self._fn, dev, self._ref,
                 rows[3] ** -0.5 if scale is None else scale, qp, qs,
                 _want("k_cache", k_cache, dt, cache, dev),
                 _want("v_cache", v_cache, dt, cache, dev),
                 _want("block_table", block_table, i32, pages, dev),
                 _want("ctx_len", ctx_len, i32, one, dev),
                 None if n_nodes is None else
                 _want("n_nodes", n_nodes, i32, one, dev),
                 None if mask is None or words[1] == 0 else
                 _want("mask", mask, torch.int64, words, dev),
                 op, *self._tail)
        return out, self.lse


def tree_attention(q, k_cache, v_cache, block_table, ctx_len, n_nodes=None,
                   mask=None, scale=None, lse: bool = False):
    """One call of TreeAttention: q [batch][N+1][Hq][D] over k_cache, v_cache
    [n_pages][Hkv][page_size][D].  Returns (out, lse or None)."""
    batch, R, Hq, D = q.shape
    n_pages, Hkv, page, _ = k_cache.shape
    h = TreeAttention(batch, R - 1, Hq, Hkv, D, n_pages, page,
                      block_table.shape[1], dtype=k_cache.dtype, lse=lse,
                      device=_dev(k_cache))
    return h.run(q, k_cache, v_cache, block_table, ctx_len, n_nodes, mask,
                 scale)


@dataclass
class CacheShare:
    """Who shares what in a round, int32: leader [batch] (the lowest request
    of the group, the request itself without one) and shared [batch] (the
    group's shared positions, 0 without one); plan: what SharedAttention
    reads, the round's lengths among it; key: the sizes it was made for."""
    leader: torch.Tensor
    shared: torch.Tensor
    plan: torch.Tensor
    key: tuple


class SharePlan:
    """Plan of the prefixes that requests of a round share, found from their
    block tables; fixed shape, with its workspace and outputs allocated once;
    run() only enqueues kernels.  least: positions that a request's pick must
    promise to save (default: 4096, times the rows of a request up to 8); the
    promise counts all requests with that page at that place, and a group
    that fewer of them form saves less.  (Attention with and without groups,
    32 heads of 128 over 400 .. 600 own positions: 8 tokens that save 1792
    positions 16.0 and 16.2 us, 7168 17.5 and 19.9; 64 tokens, 4032 32.9 and
    33.0, 16 k 34.7 and 38.0; 16 x 16 rows, 3840 26.0 and 25.3, 61 k 54 and 56;
    4 x 65 rows, 3 k 40 and 31, 12 k 56 and 52; 8 x 257 rows, 57 k 377 and
    709, 32 x 257, 63 k 669 and 756, where TreeAttention takes 374 and
    482.)"""

    def __init__(self, batch: int, N: int, n_pages: int, page_size: int,
                 max_pages: int, least: int | None = None,
                 device="cuda"):
        self.shape = CacheShape(batch, N, n_pages, page_size, max_pages, 1, 1,
                                16, PCT_BF16)
        self.device = dev = _device(device)
        self.least = 4096 * min(N + 1, 8) if least is None else least
        if not 1 <= self.least < 1 << 31:
            raise ValueError(f"least = {least} is not in 1 .. 2^31 - 1")
        self._fn, self._ref = lib().pct_cache_share, C.byref(self.shape)
        size = lib().pct_cache_share_size(self._ref)
        if size == 0:
            raise PCTError(2 if batch > 1024 else 1,
                           lib().pct_last_error().decode())
        self.ws = _workspace(lib().pct_cache_share_workspace(self._ref), dev)
        i32 = dict(dtype=torch.int32, device=dev)
        # no rows and no groups before the first run (one buffer, so that one
        # copy goes back to that)
        self._all = torch.zeros(size // 4 + 2 * batch, **i32)
        plan, leader, shared = self._all.split((size // 4, batch, batch))
        req = plan[:4 * batch].view(batch, 4)
        req[:, 1] = -1
        req[:, 3] = -1
        plan[8 * batch:10 * batch] = -1
        torch.arange(batch, out=leader)
        self._none = self._all.clone()
        self.out = CacheShare(
            leader=leader, shared=shared, plan=plan,
            key=(batch, N, n_pages, page_size, max_pages))
        o = self.out
        self._tail = tuple(C.c_void_p(x.data_ptr()) for x in (
            o.leader, o.shared, o.plan, self.ws)) + (self.ws.numel(),)

    def run(self, ctx_len, n_nodes, block_table) -> CacheShare:
        """n_nodes None = N everywhere.  The outputs are written by every
        call."""
        dev, i32 = self.device.index, torch.int32
        batch, width = self.shape.batch, self.shape.max_pages
        _enqueue(self._fn, dev, self._ref, self.least,
                 _want("ctx_len", ctx_len, i32, (batch,), dev),
                 None if n_nodes is None else
                 _want("n_nodes", n_nodes, i32, (batch,), dev),
                 _want("block_table", block_table, i32, (batch, width), dev),
                 *self._tail)
        return self.out

    def clear(self):
        """Outputs as before the first run: no rows and no groups."""
        self._all.copy_(self._none)


class SharedAttention:
    """TreeAttention that reads the keys a group of requests shares once for
    all of its rows: fixed shape, workspace and outputs allocated once; run()
    only enqueues kernels.  Its outputs carry no gradient.

    For few rows a request over long shared prefixes (16 x 65 rows over 8 k: 185
    us, TreeAttention 242).  Every row's sums go through the workspace (ws; 145
    MB there, 393 MB for 32 x 257 rows of 32 heads of 128, 2.4 GB for 128 x
    513): trees of 257 rows gain nothing (8 x 257 over 8 k 377 and 374), and
    without groups they are slower (32 x 257 over 1 k .. 4 k 811
    and 495, 128 x 513 over 256 .. 2 k 5156 and 3167)."""

    def __init__(self, batch: int, N: int, Hq: int, Hkv: int, D: int,
                 n_pages: int, page_size: int, max_pages: int,
                 dtype=torch.bfloat16, lse: bool = False, device="cuda"):
        self.dtype = dtype
        self.shape = CacheShape(batch, N, n_pages, page_size, max_pages, Hq,
                                Hkv, D, _cache_dtype(dtype))
        self.device = dev = _device(device)
        self._fn, self._ref = lib().pct_shared_attention, C.byref(self.shape)
        nbytes = lib().pct_shared_attention_workspace(self._ref)
        if nbytes == 0:
            raise PCTError(2 if batch > 1024 else 1,
                           lib().pct_last_error().decode())
        self.ws = _workspace(nbytes, dev)
        # a call writes the rows it uses: those that none has used stay zero
        self.out = torch.zeros(batch, N + 1, Hq, D, dtype=dtype, device=dev)
        self.lse = (torch.zeros(batch, N + 1, Hq, dtype=torch.float32,
                                device=dev) if lse else None)
        self._key = (batch, N, n_pages, page_size, max_pages)
        self._shapes = ((batch, N + 1, Hq, D), (n_pages, Hkv, page_size, D),
                        (batch, max_pages), (batch, N, (N + 63) // 64))
        self._op = C.c_void_p(self.out.data_ptr())
        self._tail = (None if self.lse is None else
                      C.c_void_p(self.lse.data_ptr()),
                      C.c_void_p(self.ws.data_ptr()), self.ws.numel())

    def run(self, q, k_cache, v_cache, block_table, share: CacheShare,
            mask=None, scale=None, out=None):
        """As TreeAttention.run, with the lengths of the round in `share`, as
        SharePlan.run returned it from the same block_table."""
        dev, dt, i32 = self.device.index, self.dtype, torch.int32
        rows, cache, pages, words = self._shapes
        if share.key != self._key:
            raise ValueError(f"the share plan is for sizes {share.key}, not "
                             f"{self._key}")
        if out is None:
            out, op = self.out, self._op
        else:
            op = _want("out", out, dt, rows, dev)
        qp, qs = _rows("q", q, dt, rows, dev)
        _enqueue(self._fn, dev, self._ref,
                 rows[3] ** -0.5 if scale is None else scale, qp, qs,
                 _want("k_cache", k_cache, dt, cache, dev),
                 _want("v_cache", v_cache, dt, cache, dev),
                 _want("block_table", block_table, i32, pages, dev),
                 _want("share.plan", share.plan, i32, share.plan.shape, dev),
                 None if mask is None or words[1] == 0 else
                 _want("mask", mask, torch.int64, words, dev),
                 op, *self._tail)
        return out, self.lse


def cache_commit(tau, accept_node, ctx_len, n_nodes, block_table, k_cache,
                 v_cache, out=None, N: int = 8192):
    """Keep the accepted paths: tau [batch] and accept_node [batch][B] as
    verify_accept returns them, n_nodes [batch] or None (N in every request),
    N the trees' largest size (the first accepted node outside a tree ends
    the moves), k_cache, v_cache [layers][n_pages][Hkv][page_size][D] (or one layer).
    Returns the new context lengths, in `out` when given (which may be
    ctx_len itself)."""
    dev = k_cache.get_device()
    if dev < 0:
        raise ValueError("libpctree needs device tensors")
    cache = k_cache.shape
    n_pages, Hkv, page, D = cache[-4:]
    layers = cache[0] if len(cache) == 5 else 1
    batch, B = accept_node.shape
    width = block_table.shape[-1]
    dt, i32, one = k_cache.dtype, torch.int32, (batch,)
    if out is None:
        out = torch.empty_like(ctx_len)
    sh = _shape_ref(batch, N, n_pages, page, width, Hkv, Hkv, D,
                    _cache_dtype(dt))
    _enqueue(lib().pct_cache_commit, dev, sh, layers,
             n_pages * Hkv * page * D, B, _want("tau", tau, i32, one, dev),
             _want("accept_node", accept_node, i32, (batch, B), dev),
             None if n_nodes is None else
             _want("n_nodes", n_nodes, i32, one, dev),
             _want("block_table", block_table, i32, (batch, width), dev),
             _want("ctx_len", ctx_len, i32, one, dev),
             _want("k_cache", k_cache, dt, cache, dev),
             _want("v_cache", v_cache, dt, cache, dev),
             _want("out", out, i32, one, dev))
    return out


@dataclass(frozen=True, eq=False)
class PageState:
    """The state of a cache's pages, int32: ctx_len [batch], block_table
    [batch][max_pages], n_held [batch], ring [n_pages] and ring_state [2] as
    CachePlan has them, extra [n_pages]: holders of a page beyond the first.
    The tensors are checked once, here; calls change what they hold."""
    ctx_len: torch.Tensor
    block_table: torch.Tensor
    n_held: torch.Tensor
    ring: torch.Tensor
    ring_state: torch.Tensor
    extra: torch.Tensor

    def __post_init__(self):
        batch, width = self.block_table.shape
        n_pages, dev = self.ring.numel(), self.ring.get_device()
        if dev < 0:
            raise ValueError("libpctree needs device tensors")
        shapes = ((batch,), (batch, width), (batch,), (n_pages,), (2,),
                  (n_pages,))
        names = ("ctx_len", "block_table", "n_held", "ring", "ring_state",
                 "extra")
        state = _PageState(*(
            _want(name, getattr(self, name), torch.int32, shape, dev)
            for name, shape in zip(names, shapes)))
        object.__setattr__(self, "_ref", C.byref(state))
        object.__setattr__(self, "_key", (batch, width, n_pages, dev))


class CachePages:
    """Pages that several requests hold: places freed, trimmed and forked,
    and pages in use moved to the front, for a cache of fixed shape, with the
    workspace allocated once; the calls only enqueue kernels.  Where requests
    share pages, trim() comes before CachePlan.run(), which then has nothing
    to give back."""

    def __init__(self, batch: int, n_pages: int, page_size: int,
                 max_pages: int, Hkv: int, D: int, layers: int = 1,
                 dtype=torch.bfloat16, N: int = 0, device="cuda"):
        self.shape = CacheShape(batch, N, n_pages, page_size, max_pages, Hkv,
                                Hkv, D, _cache_dtype(dtype))
        self.layers, self.dtype = layers, dtype
        self.device = dev = _device(device)
        L, self._ref = lib(), C.byref(self.shape)
        nbytes = L.pct_cache_free_workspace(self._ref)
        if nbytes == 0:
            raise PCTError(1, L.pct_last_error().decode())
        self.ws = _workspace(max(
            nbytes, L.pct_cache_compact_workspace(self._ref),
            L.pct_cache_fork_workspace(self._ref, batch)), dev)
        self._layer = n_pages * Hkv * page_size * D
        self._cache = (layers, n_pages, Hkv, page_size, D)
        self._key = (batch, max_pages, n_pages, dev.index)
        self._tail = (C.c_void_p(self.ws.data_ptr()), self.ws.numel())

    def _state(self, state: PageState):
        if state._key != self._key:
            raise ValueError("the state's (batch, max_pages, n_pages, device) "
                             f"are {state._key}, not {self._key}")
        return state._ref

    def _caches(self, k_cache, v_cache):
        dev, cache = self.device.index, self._cache
        if self.layers == 1 and k_cache.dim() == 4:
            cache = cache[1:]
        return (_want("k_cache", k_cache, self.dtype, cache, dev),
                _want("v_cache", v_cache, self.dtype, cache, dev))

    def free(self, state: PageState, places):
        """Empty places [m] int32 (entries outside the batch are left out):
        pages that nobody else holds go back to the ring."""
        dev = self.device.index
        _enqueue(lib().pct_cache_free, dev, self._ref, places.numel(),
                 _want("places", places, torch.int32, (places.numel(),), dev),
                 self._state(state), *self._tail)

    def trim(self, state: PageState, n_nodes=None):
        """Every request keeps the pages of its ctx_len + n_nodes + 1
        positions (n_nodes None: the N of this handle) and lets go of the
        rest."""
        dev = self.device.index
        _enqueue(lib().pct_cache_trim, dev, self._ref,
                 None if n_nodes is None else
                 _want("n_nodes", n_nodes, torch.int32,
                       (self.shape.batch,), dev),
                 self._state(state), *self._tail)

    def fork(self, state: PageState, src, dst, k_cache, v_cache, length=None,
             out=None):
        """Place dst[i] becomes a copy of the first length[i] positions
        (default: all) of src[i]'s context; m pairs of int32, at most as many
        as places.  k_cache, v_cache [layers][n_pages][Hkv][page_size][D]
        (or one layer).  Returns done [m] int32 (into `out` when given): 0
        where a pair is left out, since dst holds pages, src lacks some, or
        the ring has none left."""
        dev, i32, m = self.device.index, torch.int32, src.numel()
        if m > self._key[0]:
            raise PCTError(1, f"{m} pairs for {self._key[0]} places")
        if out is None:
            out = torch.empty(m, dtype=i32, device=src.device)
        kp, vp = self._caches(k_cache, v_cache)
        _enqueue(lib().pct_cache_fork, dev, self._ref, self.layers,
                 self._layer, m, _want("src", src, i32, (m,), dev),
                 _want("dst", dst, i32, (m,), dev),
                 None if length is None else
                 _want("length", length, i32, (m,), dev),
                 self._state(state), kp, vp, _want("out", out, i32, (m,), dev),
                 *self._tail)
        return out

    def compact(self, state: PageState, k_cache, v_cache, out=None):
        """Move the pages in use to the first ones of the cache; ring,
        ring_state and extra are made anew from the table, which is changed
        in place or, given `out`, written there.  Slots and share plans of
        before are void."""
        table = state.block_table if out is None else out
        kp, vp = self._caches(k_cache, v_cache)
        dev = self.device.index
        _enqueue(lib().pct_cache_compact, dev, self._ref, self.layers,
                 self._layer, self._state(state),
                 _want("out", table, torch.int32, self._key[:2], dev), kp, vp,
                 *self._tail)
        return table


class PagedCache:
    """A paged key-value cache of a serving batch: k, v
    [layers][n_pages][Hkv][page_size][D], the block table, the pages held,
    the free ring and the context lengths of `batch` places.

    A round: rows = plan(n_nodes, depth); in each layer write(layer, k, v)
    and attend(layer, q, mask); then commit(tau, accept_node).  A place is
    emptied by setting its ctx_len to 0 and its n_nodes to -1 for one plan.
    Before the first plan nothing is written, attended or kept.

    A request that the free ring cannot serve (rows.missing > 0) waits: it is
    not attended, and commit leaves its length and its cache as they are
    whatever tau and accept_node say.  It keeps its root for a later round.
    n_nodes is what the last plan was given, n_served what was served of it.

    share: requests may hold the same pages (extra counts their holders).
    fork() makes a place a copy of another's context, free() empties places,
    compact() moves the pages in use to the front, all between a commit and
    the next plan (until then nothing is written, rotated, attended or kept,
    and nobody shares), and
    attend reads what requests share once for all of them, if that promises to
    save `least` positions (SharePlan).  batch is at most 1024 then.  All
    rounds attend by SharedAttention, with its workspace; large trees have
    faster rows of a TreeAttention on block_table, ctx_len and n_served.
    """

    def __init__(self, batch: int, N: int, n_pages: int, page_size: int,
                 max_pages: int, Hq: int, Hkv: int, D: int, layers: int = 1,
                 dtype=torch.bfloat16, share: bool = False,
                 least: int | None = None, device="cuda"):
        dev = _device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.k = torch.zeros(layers, n_pages, Hkv, page_size, D, dtype=dtype,
                             device=dev)
        self.v = torch.zeros_like(self.k)
        self.block_table = torch.full((batch, max_pages), -1, **i32)
        self.n_held = torch.zeros(batch, **i32)
        self.ring = torch.arange(n_pages, **i32)
        self.ring_state = torch.tensor([0, n_pages], **i32)
        self.ctx_len = torch.zeros(batch, **i32)
        self._plan = CachePlan(batch, N, n_pages, page_size, max_pages,
                               device=dev)
        self.n_nodes = None
        self.n_served = self._plan.out.n_served
        sizes = (batch, N, Hq, Hkv, D, n_pages, page_size, max_pages)
        self.share = None
        if share:
            self.extra = torch.zeros(n_pages, **i32)
            self._pages = CachePages(batch, n_pages, page_size, max_pages,
                                     Hkv, D, layers=layers, dtype=dtype, N=N,
                                     device=dev)
            self._share = SharePlan(batch, N, n_pages, page_size, max_pages,
                                    least=least, device=dev)
            self.share = self._share.out
            self._attend = SharedAttention(*sizes, dtype=dtype, device=dev)
        else:
            self._attend = TreeAttention(*sizes, dtype=dtype, device=dev)

    def _state(self) -> PageState:
        if self.share is None:
            raise ValueError("the cache was made without share=True")
        return PageState(self.ctx_len, self.block_table, self.n_held,
                         self.ring, self.ring_state, self.extra)

    def _void(self):
        """Until the next plan there are no rows and no groups."""
        self._plan.out.slot.fill_(-1)
        self._plan.out.pos.fill_(-1)
        self.n_served.fill_(-1)
        self._share.clear()

    def fork(self, src, dst, length=None):
        """Place dst[i] becomes a copy of the first length[i] (default: all)
        positions of src[i]'s context (CachePages.fork); returns done [m]."""
        state = self._state()
        done = self._pages.fork(state, src, dst, self.k, self.v,
                                length=length)
        self._void()
        return done

    def free(self, places):
        """Empty places [m] int32; entries outside the batch are left out."""
        state = self._state()
        self._pages.free(state, places)
        self._void()

    def compact(self):
        """Move the pages in use to the first ones of the cache; there are
        n_pages - ring_state[1] of them."""
        state = self._state()
        self._pages.compact(state, self.k, self.v)
        self._void()

    def plan(self, n_nodes=None, depth=None) -> CacheRows:
        if self.share is not None:
            # (what the plan refuses is refused before pages are let go)
            self._plan._depth(depth)
            if n_nodes is not None and \
                    n_nodes.data_ptr() == self.n_served.data_ptr():
                raise PCTError(1, "n_served overlaps n_nodes or ctx_len")
            # (pages that others hold must not go back to the ring)
            self._pages.trim(self._state(), n_nodes)
        rows = self._plan.run(self.ctx_len, n_nodes, self.block_table,
                              self.n_held, self.ring, self.ring_state,
                              depth=depth)
        self.n_nodes = n_nodes
        if self.share is not None:
            self._share.run(self.ctx_len, self.n_served, self.block_table)
        return rows

    def write(self, layer: int, k, v):
        cache_write(k, v, self._plan.out.slot, self.k[layer], self.v[layer])

    def write_rotary(self, layer: int, rotary: Rotary, q, k, v,
                     q_weight=None, k_weight=None, eps: float = 1e-6,
                     out=None):
        """write() of a layer whose queries and keys are normalised (with
        weights) and rotated to the rows' places on the way; returns the
        rotated queries (cache_write_rotary), by default a new tensor of zeros
        in each call: give `out` in the layers of a round."""
        o = self._plan.out
        return cache_write_rotary(rotary, q, k, v, o.pos, o.slot,
                                  self.k[layer], self.v[layer],
                                  q_weight=q_weight, k_weight=k_weight,
                                  eps=eps, out=out)

    def attend(self, layer: int, q, mask=None, scale=None, out=None):
        """The layer's attention, in `out` when given, else in a tensor that
        every call without `out` writes, whatever its layer.  Unused rows,
        and those of requests that wait, are left as they were there."""
        of = ((self.ctx_len, self.n_served) if self.share is None
              else (self.share,))
        return self._attend.run(q, self.k[layer], self.v[layer],
                                self.block_table, *of, mask=mask, scale=scale,
                                out=out)[0]

    def commit(self, tau, accept_node):
        return cache_commit(tau, accept_node, self.ctx_len, self.n_served,
                            self.block_table, self.k, self.v,
                            out=self.ctx_len, N=self._plan.shape.N)


def bf16_tensor(bits, device="cuda") -> torch.Tensor:
    """uint16 bf16 bit patterns (numpy) -> a bfloat16 device tensor."""
    import numpy as np
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.to(device).view(torch.bfloat16)
