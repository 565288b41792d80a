// api_cache.hip -- the C-ABI of the paged key-value cache: argument checks
// and launches of the page plan, row writes, tree attention and the commit
// of accepted paths.
#include "api_cache.h"

using namespace pct;

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
  pct_cache_shape sh;
  if (shape) {
    // the block table is not read: its width does not matter here
    sh = *shape;
    sh.max_pages = 1;
    shape = &sh;
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
  if (!ctx_len)
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  AttendArgs a{};
  st = attend_args(shape, scale, q, q_row_stride, k_cache, v_cache,
                   block_table, ctx_len, n_nodes, mask, out, lse, a);
  if (st != PCT_OK) return st;
  const size_t need = tree_attention_workspace(*shape);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(PCT_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (need > 0 && !aligned16(workspace))
    return fail(PCT_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
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
