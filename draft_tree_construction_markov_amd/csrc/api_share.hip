// api_share.hip -- the C-ABI of shared prefixes: the share plan of a round and
// attention that reads shared keys once.
#include <math.h>

#include "api_cache.h"

using namespace pct;

namespace {

pct_status check_share(const pct_cache_shape* sh) {
  const pct_status st = check_pages(sh);
  if (st != PCT_OK) return st;
  if (sh->batch > kMaxShareBatch)
    return fail(PCT_ERR_UNSUPPORTED, "batch = %d exceeds %d", sh->batch,
                kMaxShareBatch);
  return PCT_OK;
}

// packed rows and row tiles are counted in 32 bits
pct_status check_packed(const pct_cache_shape* sh) {
  if ((int64_t)sh->batch * (sh->N + 1) * (sh->Hq / sh->Hkv) > 1 << 30)
    return fail(PCT_ERR_UNSUPPORTED,
                "batch * (N + 1) * Hq / Hkv exceeds 2^30");
  return PCT_OK;
}

ShareView view_of(const pct_cache_shape* sh, const void* share) {
  ShareView v{};
  v.req = static_cast<int4*>(const_cast<void*>(share));
  v.groups = v.req + sh->batch;
  v.group_of = reinterpret_cast<int2*>(v.groups + sh->batch);
  v.totals = reinterpret_cast<float*>(v.group_of + sh->batch);
  v.rows = reinterpret_cast<int32_t*>(v.totals + 4);
  return v;
}

size_t share_size(const pct_cache_shape* sh) {
  return 4 * sizeof(float) +
         (size_t)sh->batch * (2 * sizeof(int4) + sizeof(int2)) +
         (size_t)sh->batch * (sh->N + 1) * sizeof(int32_t);
}

size_t share_workspace(const pct_cache_shape* sh) {
  return (size_t)sh->batch * ((size_t)share_blocks(*sh) * sizeof(uint64_t) +
                              2 * sizeof(int32_t));
}

}  // namespace

extern "C" {

size_t pct_cache_share_size(const pct_cache_shape* shape) {
  return check_share(shape) == PCT_OK ? share_size(shape) : 0;
}

size_t pct_cache_share_workspace(const pct_cache_shape* shape) {
  return check_share(shape) == PCT_OK ? share_workspace(shape) : 0;
}

pct_status pct_cache_share(const pct_cache_shape* shape, int32_t least,
                           const int32_t* ctx_len, const int32_t* n_nodes,
                           const int32_t* block_table, int32_t* leader,
                           int32_t* shared, void* share, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const pct_status st = check_share(shape);
  if (st != PCT_OK) return st;
  if (least < 1) return fail(PCT_ERR_INVALID_ARG, "least must be positive");
  if (!ctx_len || !block_table || !leader || !shared || !share)
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  if (!aligned16(share))
    return fail(PCT_ERR_INVALID_ARG, "share must be 16-byte aligned");
  const size_t need = share_workspace(shape);
  if (!workspace || workspace_bytes < need)
    return fail(PCT_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (!aligned16(workspace))
    return fail(PCT_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  const size_t n = 4 * (size_t)shape->batch;
  const struct {
    const void* p;
    size_t bytes;
  } all[] = {{leader, n},
             {shared, n},
             {share, share_size(shape)},
             {workspace, need},
             {ctx_len, n},
             {n_nodes, n},
             {block_table, n * shape->max_pages}};
  // (the first four are written)
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 7; ++j)
      if (bytes_meet(all[i].p, all[i].bytes, all[j].p, all[j].bytes))
        return fail(PCT_ERR_INVALID_ARG,
                    "leader, shared, share or the workspace overlap each "
                    "other or an input");
  ShareArgs a{};
  a.g = geom(shape, block_table, ctx_len, n_nodes);
  a.least = least;
  a.best = static_cast<uint64_t*>(workspace);
  a.blocks = share_blocks(*shape);
  a.place =
      reinterpret_cast<int32_t*>(a.best + (size_t)a.blocks * shape->batch);
  a.joined = a.place + shape->batch;
  a.leader = leader;
  a.shared = shared;
  a.view = view_of(shape, share);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  {
    ProfScope ps(PROF_SHARE, shape->batch, s);
    e = launch_share(a, s);
  }
  if (e != hipSuccess) return hip_fail(e, "share plan kernel");
  return PCT_OK;
}

size_t pct_shared_attention_workspace(const pct_cache_shape* shape) {
  if (check_share(shape) != PCT_OK || check_heads(shape, true) != PCT_OK ||
      check_packed(shape) != PCT_OK)
    return 0;
  return shared_attention_workspace(*shape);
}

pct_status pct_shared_attention(const pct_cache_shape* shape, float scale,
                                const void* q, int64_t q_row_stride,
                                const void* k_cache, const void* v_cache,
                                const int32_t* block_table, const void* share,
                                const uint64_t* mask, void* out, float* lse,
                                void* workspace, size_t workspace_bytes,
                                void* stream) {
  pct_status st = check_share(shape);
  if (st != PCT_OK) return st;
  st = check_heads(shape, true);
  if (st != PCT_OK) return st;
  if (!share) return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  if (!aligned16(share))
    return fail(PCT_ERR_INVALID_ARG, "share must be 16-byte aligned");
  // (the lengths are the share plan's)
  AttendArgs a{};
  st = attend_args(shape, scale, q, q_row_stride, k_cache, v_cache,
                   block_table, nullptr, nullptr, mask, out, lse, a);
  if (st != PCT_OK) return st;
  st = check_packed(shape);
  if (st != PCT_OK) return st;
  const size_t need = shared_attention_workspace(*shape);
  if (!workspace || workspace_bytes < need)
    return fail(PCT_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (!aligned16(workspace))
    return fail(PCT_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  a.share = view_of(shape, share);
  const hipError_t e =
      launch_shared_attention(a, workspace, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "shared attention kernel");
  return PCT_OK;
}

}  // extern "C"
