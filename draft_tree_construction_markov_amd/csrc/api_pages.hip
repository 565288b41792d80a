// api_pages.hip -- the C-ABI of pages that several requests hold: free, trim,
// fork and compact.
#include "api_cache.h"

using namespace pct;

namespace {

// Arrays of a call, for the checks of overlap.
struct Span {
  const int32_t* p;
  int64_t n;
};

struct StateSpans {
  Span all[6];
};
StateSpans spans_of(const pct_cache_shape* sh, const pct_page_state* st) {
  return {{{st->ctx_len, sh->batch},
           {st->block_table, (int64_t)sh->batch * sh->max_pages},
           {st->n_held, sh->batch},
           {st->ring, sh->n_pages},
           {st->ring_state, 2},
           {st->extra, sh->n_pages}}};
}

pct_status check_state(const pct_cache_shape* sh, const pct_page_state* st) {
  // (pages are counted in 32 bits, past the last one of a scan)
  if (sh->n_pages > 1 << 30)
    return fail(PCT_ERR_UNSUPPORTED, "n_pages = %d exceeds 2^30", sh->n_pages);
  if (!st) return fail(PCT_ERR_INVALID_ARG, "state is NULL");
  const StateSpans x = spans_of(sh, st);
  for (const Span& y : x.all)
    if (!y.p) return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  for (int i = 0; i < 6; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(x.all[i].p, x.all[i].n, x.all[j].p, x.all[j].n))
        return fail(PCT_ERR_INVALID_ARG, "arrays of the state overlap");
  return PCT_OK;
}

// whether n values from x on meet an array of the state
bool meets_state(const pct_cache_shape* sh, const pct_page_state* st,
                 const int32_t* x, int64_t n) {
  for (const Span& y : spans_of(sh, st).all)
    if (overlap(x, n, y.p, y.n)) return true;
  return false;
}

// The workspace holds what kernels of a call leave for the next ones: it must
// not meet the state, which the call changes, nor its other arrays.
template <int N>
pct_status check_workspace(const void* ws, size_t have, size_t need,
                           const pct_cache_shape* sh, const pct_page_state* st,
                           const Span (&more)[N]) {
  if (!ws || have < need)
    return fail(PCT_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (!aligned16(ws))
    return fail(PCT_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  const auto meets = [&](const Span& y) {
    return bytes_meet(ws, need, y.p, 4 * (size_t)y.n);
  };
  bool met = false;
  for (const Span& y : spans_of(sh, st).all) met = met || meets(y);
  for (const Span& y : more) met = met || meets(y);
  return met ? fail(PCT_ERR_INVALID_ARG,
                    "workspace overlaps the state or another array")
             : PCT_OK;
}

pct_status check_caches(const pct_cache_shape* sh, int layers,
                        int64_t layer_stride, const void* k, const void* v) {
  const pct_status st = check_heads(sh, false);
  if (st != PCT_OK) return st;
  if (layers < 1 || layers > 1024)
    return fail(PCT_ERR_INVALID_ARG, "need 1 <= layers <= 1024");
  const int64_t layer =
      (int64_t)sh->n_pages * sh->Hkv * sh->page_size * sh->D;
  if (layer_stride % 8 != 0 || (layers > 1 && layer_stride < layer))
    return fail(PCT_ERR_INVALID_ARG,
                "layer_stride must be a multiple of 8 and hold a layer");
  if (!k || !v) return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  if (!aligned16(k) || !aligned16(v))
    return fail(PCT_ERR_INVALID_ARG, "caches must be 16-byte aligned");
  return PCT_OK;
}

PagesArgs pages_args(const pct_cache_shape* sh, const pct_page_state* st,
                     const int32_t* n_nodes) {
  PagesArgs a{};
  a.g = geom(sh, nullptr, nullptr, n_nodes);
  a.ctx = st->ctx_len;
  a.table = st->block_table;
  a.held = st->n_held;
  a.ring = st->ring;
  a.ring_state = st->ring_state;
  a.extra = st->extra;
  a.m = sh->batch;
  return a;
}

pct_status release(const PagesArgs& a, hipStream_t s) {
  hipError_t e;
  {
    ProfScope ps(PROF_RELEASE, a.m, s);
    e = launch_release(a, s);
  }
  return e == hipSuccess ? PCT_OK : hip_fail(e, "page release kernel");
}

size_t fork_workspace(int batch, int m) {
  return (size_t)m * sizeof(int4) + (size_t)batch * sizeof(int32_t);
}

}  // namespace

extern "C" {

size_t pct_cache_free_workspace(const pct_cache_shape* shape) {
  return check_pages(shape) == PCT_OK ? release_workspace(*shape) : 0;
}

pct_status pct_cache_free(const pct_cache_shape* shape, int32_t m,
                          const int32_t* places, const pct_page_state* state,
                          void* workspace, size_t workspace_bytes,
                          void* stream) {
  pct_status st = check_pages(shape);
  if (st != PCT_OK) return st;
  if (m < 0) return fail(PCT_ERR_INVALID_ARG, "m = %d is negative", m);
  if (m > 65535)
    return fail(PCT_ERR_UNSUPPORTED, "m = %d exceeds 65535", m);
  if ((st = check_state(shape, state)) != PCT_OK) return st;
  if (m > 0 && !places)
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  if (meets_state(shape, state, places, m))
    return fail(PCT_ERR_INVALID_ARG, "places overlaps the state");
  const Span more[] = {{places, m}};
  st = check_workspace(workspace, workspace_bytes, release_workspace(*shape),
                       shape, state, more);
  if (st != PCT_OK || m == 0) return st;
  PagesArgs a = pages_args(shape, state, nullptr);
  a.m = m;
  a.places = places;
  a.count = static_cast<int32_t*>(workspace);
  return release(a, static_cast<hipStream_t>(stream));
}

pct_status pct_cache_trim(const pct_cache_shape* shape, const int32_t* n_nodes,
                          const pct_page_state* state, void* workspace,
                          size_t workspace_bytes, void* stream) {
  pct_status st = check_pages(shape);
  if (st != PCT_OK) return st;
  if ((st = check_state(shape, state)) != PCT_OK) return st;
  if (meets_state(shape, state, n_nodes, shape->batch))
    return fail(PCT_ERR_INVALID_ARG, "n_nodes overlaps the state");
  const Span more[] = {{n_nodes, shape->batch}};
  st = check_workspace(workspace, workspace_bytes, release_workspace(*shape),
                       shape, state, more);
  if (st != PCT_OK) return st;
  PagesArgs a = pages_args(shape, state, n_nodes);
  a.count = static_cast<int32_t*>(workspace);
  return release(a, static_cast<hipStream_t>(stream));
}

size_t pct_cache_fork_workspace(const pct_cache_shape* shape, int32_t m) {
  if (check_pages(shape) != PCT_OK || m < 0 || m > 65535) return 0;
  return fork_workspace(shape->batch, m);
}

pct_status pct_cache_fork(const pct_cache_shape* shape, int32_t layers,
                          int64_t layer_stride, int32_t m, const int32_t* src,
                          const int32_t* dst, const int32_t* length,
                          const pct_page_state* state, void* k_cache,
                          void* v_cache, int32_t* done, void* workspace,
                          size_t workspace_bytes, void* stream) {
  pct_status st = check_pages(shape);
  if (st != PCT_OK) return st;
  if ((st = check_caches(shape, layers, layer_stride, k_cache, v_cache)) !=
      PCT_OK)
    return st;
  if (m < 0) return fail(PCT_ERR_INVALID_ARG, "m = %d is negative", m);
  if (m > 65535)
    return fail(PCT_ERR_UNSUPPORTED, "m = %d exceeds 65535", m);
  if ((st = check_state(shape, state)) != PCT_OK) return st;
  if (m > 0 && (!src || !dst || !done))
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  if (meets_state(shape, state, src, m) || meets_state(shape, state, dst, m) ||
      meets_state(shape, state, length, m) ||
      meets_state(shape, state, done, m) || overlap(done, m, src, m) ||
      overlap(done, m, dst, m) || overlap(done, m, length, m))
    return fail(PCT_ERR_INVALID_ARG,
                "src, dst, length or done overlap the state or each other");
  const Span more[] = {{src, m}, {dst, m}, {length, m}, {done, m}};
  st = check_workspace(workspace, workspace_bytes,
                       fork_workspace(shape->batch, m), shape, state, more);
  if (st != PCT_OK || m == 0) return st;
  ForkArgs f{};
  f.a = pages_args(shape, state, nullptr);
  f.a.m = m;
  f.a.layers = layers;
  f.a.layer_stride = layer_stride / 8;
  f.a.kc = static_cast<uint4*>(k_cache);
  f.a.vc = static_cast<uint4*>(v_cache);
  f.src = src;
  f.dst = dst;
  f.length = length;
  f.done = done;
  f.req = static_cast<int4*>(workspace);
  f.claim = reinterpret_cast<int32_t*>(f.req + m);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  {
    ProfScope ps(PROF_FORK, m, s);
    e = launch_fork(f, s);
  }
  if (e != hipSuccess) return hip_fail(e, "cache fork kernel");
  return PCT_OK;
}

size_t pct_cache_compact_workspace(const pct_cache_shape* shape) {
  return check_pages(shape) == PCT_OK ? compact_workspace(*shape) : 0;
}

pct_status pct_cache_compact(const pct_cache_shape* shape, int32_t layers,
                             int64_t layer_stride, const pct_page_state* state,
                             int32_t* table_out, void* k_cache, void* v_cache,
                             void* workspace, size_t workspace_bytes,
                             void* stream) {
  pct_status st = check_pages(shape);
  if (st != PCT_OK) return st;
  if ((st = check_caches(shape, layers, layer_stride, k_cache, v_cache)) !=
      PCT_OK)
    return st;
  if ((st = check_state(shape, state)) != PCT_OK) return st;
  if (!table_out)
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  if (table_out != state->block_table &&
      meets_state(shape, state, table_out,
                  (int64_t)shape->batch * shape->max_pages))
    return fail(PCT_ERR_INVALID_ARG, "table_out overlaps the state");
  const Span more[] = {{table_out, (int64_t)shape->batch * shape->max_pages}};
  st = check_workspace(workspace, workspace_bytes, compact_workspace(*shape),
                       shape, state, more);
  if (st != PCT_OK) return st;
  CompactArgs c{};
  c.a = pages_args(shape, state, nullptr);
  c.a.layers = layers;
  c.a.layer_stride = layer_stride / 8;
  c.a.kc = static_cast<uint4*>(k_cache);
  c.a.vc = static_cast<uint4*>(v_cache);
  c.table_out = table_out;
  const size_t P = (size_t)shape->n_pages;
  c.info = static_cast<int32_t*>(workspace);
  c.hole = c.info + 4;
  c.high = c.hole + P;
  c.rank = c.high + P;
  c.a.count = c.rank + P;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  {
    ProfScope ps(PROF_COMPACT, shape->n_pages, s);
    e = launch_compact(c, s);
  }
  if (e != hipSuccess) return hip_fail(e, "cache compaction kernel");
  return PCT_OK;
}

}  // extern "C"
