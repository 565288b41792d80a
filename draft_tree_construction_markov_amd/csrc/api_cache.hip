// api_cache.hip -- the C-ABI of the paged key-value cache: argument checks
// and launches of the page plan, row writes, tree attention and the commit
// of accepted paths.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "pct_cache.h"

using namespace pct;

namespace {

pct_status fail(pct_status st, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return set_error(st, msg);
}

pct_status hip_fail(hipError_t e, const char* what) {
  return fail(PCT_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// arrays of n and m values that share memory (a null pointer has none)
bool overlap(const int32_t* x, int64_t n, const int32_t* y, int64_t m) {
  const uintptr_t p = (uintptr_t)x, q = (uintptr_t)y;
  return x && y && p < q + 4 * (uintptr_t)m && q < p + 4 * (uintptr_t)n;
}

int log2_of(int x) { return 31 - __builtin_clz((unsigned)x); }

pct_status check_pages(const pct_cache_shape* sh) {
  if (!sh) return fail(PCT_ERR_INVALID_ARG, "shape is NULL");
  if (sh->batch < 1 || sh->N < 0 || sh->N > 8192 || sh->n_pages < 1 ||
      sh->max_pages < 1)
    return fail(PCT_ERR_INVALID_ARG,
                "need batch, n_pages, max_pages >= 1 and 0 <= N <= 8192");
  if (sh->page_size < 1 || sh->page_size > 1024 ||
      (sh->page_size & (sh->page_size - 1)) != 0)
    return fail(PCT_ERR_INVALID_ARG,
                "page_size = %d is not a power of two up to 1024",
                sh->page_size);
  if ((int64_t)sh->max_pages * sh->page_size > kMaxTokens)
    return fail(PCT_ERR_INVALID_ARG, "max_pages * page_size exceeds 2^30");
  if (sh->batch > 65535)
    return fail(PCT_ERR_UNSUPPORTED, "batch = %d exceeds 65535", sh->batch);
  return PCT_OK;
}

pct_status check_heads(const pct_cache_shape* sh, bool queries) {
  if (sh->Hkv < 1 || sh->Hkv > 1024)
    return fail(PCT_ERR_INVALID_ARG, "need 1 <= Hkv <= 1024");
  if (queries && (sh->Hq < 1 || sh->Hq > 1024 || sh->Hq % sh->Hkv != 0))
    return fail(PCT_ERR_INVALID_ARG,
                "Hq = %d is not a multiple of Hkv = %d up to 1024", sh->Hq,
                sh->Hkv);
  if (sh->D < 16 || sh->D > 256 || sh->D % 16 != 0)
    return fail(PCT_ERR_INVALID_ARG,
                "D = %d is not a multiple of 16 up to 256", sh->D);
  if (sh->dtype != PCT_BF16 && sh->dtype != PCT_F16)
    return fail(PCT_ERR_INVALID_ARG, "the cache holds bf16 or fp16");
  return PCT_OK;
}

PageGeom geom(const pct_cache_shape* sh, const int32_t* table,
              const int32_t* ctx_len, const int32_t* n_nodes) {
  PageGeom g{};
  g.batch = sh->batch;
  g.N = sh->N;
  g.n_pages = sh->n_pages;
  g.max_pages = sh->max_pages;
  g.shift = log2_of(sh->page_size);
  g.Hkv = sh->Hkv;
  g.D = sh->D;
  g.table = table;
  g.ctx_len = ctx_len;
  g.n_nodes = n_nodes;
  return g;
}

}  // namespace

extern "C" {

size_t pct_cache_plan_workspace(int32_t batch) {
  return batch < 1 || batch > 65535 ? 0 : ((size_t)batch + 1) * sizeof(int4);
}

pct_status pct_cache_plan_served(
    const pct_cache_shape* shape, const int32_t* ctx_len,
    const int32_t* n_nodes, const int32_t* depth, int32_t* block_table,
    int32_t* n_held, int32_t* ring, int32_t* ring_state, int64_t* slot,
    int32_t* pos, int32_t* missing, int32_t* n_served, void* workspace,
    size_t workspace_bytes, void* stream) {
  pct_status st = check_pages(shape);
  if (st != PCT_OK) return st;
  if (!ctx_len || !block_table || !n_held || !ring || !ring_state || !slot ||
      !missing || (pos && shape->N > 0 && !depth))
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  if (overlap(n_served, shape->batch, n_nodes, shape->batch) ||
      overlap(n_served, shape->batch, ctx_len, shape->batch))
    return fail(PCT_ERR_INVALID_ARG, "n_served overlaps n_nodes or ctx_len");
  const size_t need = pct_cache_plan_workspace(shape->batch);
  if (!workspace || workspace_bytes < need)
    return fail(PCT_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (!aligned16(workspace))
    return fail(PCT_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  PlanArgs a{};
  a.g = geom(shape, nullptr, ctx_len, n_nodes);
  a.depth = depth;
  a.table = block_table;
  a.held = n_held;
  a.ring = ring;
  a.ring_state = ring_state;
  a.slot = slot;
  a.pos = pos;
  a.missing = missing;
  a.served = n_served;
  a.req = static_cast<int4*>(workspace);
  a.ring0 = reinterpret_cast<int2*>(a.req + shape->batch);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  {
    ProfScope ps(PROF_PLAN, shape->batch, s);
    e = launch_cache_plan(a, s);
  }
  if (e != hipSuccess) return hip_fail(e, "cache plan kernel");
  return PCT_OK;
}

pct_status pct_cache_plan(const pct_cache_shape* shape,
                          const int32_t* ctx_len, const int32_t* n_nodes,
                          const int32_t* depth, int32_t* block_table,
                          int32_t* n_held, int32_t* ring,
                          int32_t* ring_state, int64_t* slot, int32_t* pos,
                          int32_t* missing, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return pct_cache_plan_served(shape, ctx_len, n_nodes, depth, block_table,
                               n_held, ring, ring_state, slot, pos, missing,
                               nullptr, workspace, workspace_bytes, stream);
}

pct_status pct_cache_write(const pct_cache_shape* shape, const void* k,
                           int64_t k_row_stride, const void* v,
                           int64_t v_row_stride, const int64_t* slot,
                           void* k_cache, void* v_cache, void* stream) {
  if (shape && shape->max_pages < 1) {
    // the block table is not read: its width does not matter here
    pct_cache_shape sh = *shape;
    sh.max_pages = 1;
    return pct_cache_write(&sh, k, k_row_stride, v, v_row_stride, slot,
                           k_cache, v_cache, stream);
  }
  pct_status st = check_pages(shape);
  if (st != PCT_OK) return st;
  st = check_heads(shape, false);
  if (st != PCT_OK) return st;
  if (!k || !v || !slot || !k_cache || !v_cache)
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  const int64_t row = (int64_t)shape->Hkv * shape->D;
  if (k_row_stride < row || v_row_stride < row || k_row_stride % 8 != 0 ||
      v_row_stride % 8 != 0)
    return fail(PCT_ERR_INVALID_ARG,
                "row strides must be multiples of 8 and at least Hkv * D");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) ||
      !aligned16(v_cache))
    return fail(PCT_ERR_INVALID_ARG, "rows and caches must be 16-byte aligned");
  WriteArgs a{};
  a.rows = (int64_t)shape->batch * (shape->N + 1);
  a.shift = log2_of(shape->page_size);
  a.n_slots = (int64_t)shape->n_pages << a.shift;
  a.Hkv = shape->Hkv;
  a.D = shape->D;
  a.k = static_cast<const uint4*>(k);
  a.v = static_cast<const uint4*>(v);
  a.ks = k_row_stride / 8;
  a.vs = v_row_stride / 8;
  a.slot = slot;
  a.kc = static_cast<uint4*>(k_cache);
  a.vc = static_cast<uint4*>(v_cache);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  {
    ProfScope ps(PROF_CACHE_WRITE, a.rows, s);
    e = launch_cache_write(a, s);
  }
  if (e != hipSuccess) return hip_fail(e, "cache write kernel");
  return PCT_OK;
}

size_t pct_tree_attention_workspace(const pct_cache_shape* shape) {
  if (check_pages(shape) != PCT_OK || check_heads(shape, true) != PCT_OK)
    return 0;
  return tree_attention_workspace(*shape);
}

pct_status pct_tree_attention(const pct_cache_shape* shape, float scale,
                              const void* q, int64_t q_row_stride,
                              const void* k_cache, const void* v_cache,
                              const int32_t* block_table,
                              const int32_t* ctx_len, const int32_t* n_nodes,
                              const uint64_t* mask, void* out, float* lse,
                              void* workspace, size_t workspace_bytes,
                              void* stream) {
  pct_status st = check_pages(shape);
  if (st != PCT_OK) return st;
  st = check_heads(shape, true);
  if (st != PCT_OK) return st;
  if (!q || !k_cache || !v_cache || !block_table || !ctx_len || !out)
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  // (infinite for the largest scales: every score would be infinite or NaN)
  const float c = fabsf(scale) * 1.44269504f;
  if (!isfinite(c))
    return fail(PCT_ERR_INVALID_ARG, "scale * log2(e) must be finite");
  if (q_row_stride < (int64_t)shape->Hq * shape->D || q_row_stride % 8 != 0)
    return fail(PCT_ERR_INVALID_ARG,
                "q_row_stride must be a multiple of 8 and at least Hq * D");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(out))
    return fail(PCT_ERR_INVALID_ARG,
                "q, caches and out must be 16-byte aligned");
  const size_t need = tree_attention_workspace(*shape);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(PCT_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (need > 0 && !aligned16(workspace))
    return fail(PCT_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  AttendArgs a{};
  a.g = geom(shape, block_table, ctx_len, n_nodes);
  a.Hq = shape->Hq;
  a.G = shape->Hq / shape->Hkv;
  a.bf16 = shape->dtype == PCT_BF16;
  a.c = scale == 0.f ? 1.f : c;
  a.qand = scale == 0.f ? 0u : ~0u;
  a.qxor = scale < 0.f ? 0x80008000u : 0u;
  a.q = q;
  a.qs = q_row_stride;
  a.kc = k_cache;
  a.vc = v_cache;
  a.mask = shape->N > 0 ? mask : nullptr;
  a.words = (shape->N + 63) / 64;
  a.out = out;
  a.lse = lse;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = launch_tree_attention(a, workspace, s);
  if (e != hipSuccess) return hip_fail(e, "tree attention kernel");
  return PCT_OK;
}

pct_status pct_cache_commit(const pct_cache_shape* shape, int32_t layers,
                            int64_t layer_stride, int32_t B,
                            const int32_t* tau, const int32_t* accept_node,
                            const int32_t* n_nodes,
                            const int32_t* block_table,
                            const int32_t* ctx_len, void* k_cache,
                            void* v_cache, int32_t* ctx_out, void* stream) {
  pct_status st = check_pages(shape);
  if (st != PCT_OK) return st;
  st = check_heads(shape, false);
  if (st != PCT_OK) return st;
  if (layers < 1 || layers > 1024 || B < 1 || B > 8192)
    return fail(PCT_ERR_INVALID_ARG,
                "need 1 <= layers <= 1024 and 1 <= B <= 8192");
  if (!tau || !accept_node || !block_table || !ctx_len || !k_cache ||
      !v_cache || !ctx_out)
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  const int64_t layer =
      (int64_t)shape->n_pages * shape->Hkv * shape->page_size * shape->D;
  if (layer_stride % 8 != 0 || (layers > 1 && layer_stride < layer))
    return fail(PCT_ERR_INVALID_ARG,
                "layer_stride must be a multiple of 8 and hold a layer");
  const int64_t n = shape->batch;
  if (ctx_out != ctx_len && overlap(ctx_out, n, ctx_len, n))
    return fail(PCT_ERR_INVALID_ARG, "ctx_out overlaps ctx_len");
  // (workgroups of a request read these after one of them wrote its length)
  if (overlap(ctx_out, n, tau, n) || overlap(ctx_out, n, n_nodes, n) ||
      overlap(ctx_out, n, accept_node, n * B))
    return fail(PCT_ERR_INVALID_ARG,
                "ctx_out overlaps tau, accept_node or n_nodes");
  if (!aligned16(k_cache) || !aligned16(v_cache))
    return fail(PCT_ERR_INVALID_ARG, "caches must be 16-byte aligned");
  CommitArgs a{};
  a.g = geom(shape, block_table, ctx_len, n_nodes);
  a.layers = layers;
  a.B = B;
  a.layer_stride = layer_stride / 8;
  a.tau = tau;
  a.accept = accept_node;
  a.kc = static_cast<uint4*>(k_cache);
  a.vc = static_cast<uint4*>(v_cache);
  a.ctx_out = ctx_out;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  {
    ProfScope ps(PROF_COMMIT, shape->batch, s);
    e = launch_cache_commit(a, s);
  }
  if (e != hipSuccess) return hip_fail(e, "cache commit kernel");
  return PCT_OK;
}

}  // extern "C"
