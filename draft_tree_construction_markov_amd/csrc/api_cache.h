// api_cache.h -- argument checks that the cache's entry points share.
#pragma once

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "pct_cache.h"

namespace pct {

inline pct_status fail(pct_status st, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return set_error(st, msg);
}

inline pct_status hip_fail(hipError_t e, const char* what) {
  return fail(PCT_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// memory of n bytes from x on and of m bytes from y on meet (a null pointer
// has none)
inline bool bytes_meet(const void* x, size_t n, const void* y, size_t m) {
  const uintptr_t p = (uintptr_t)x, q = (uintptr_t)y;
  return x && y && p < q + m && q < p + n;
}
// arrays of n and m values that share memory
inline bool overlap(const int32_t* x, int64_t n, const int32_t* y, int64_t m) {
  return bytes_meet(x, 4 * (size_t)n, y, 4 * (size_t)m);
}

inline int log2_of(int x) { return 31 - __builtin_clz((unsigned)x); }

inline pct_status check_pages(const pct_cache_shape* sh) {
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

inline pct_status check_heads(const pct_cache_shape* sh, bool queries) {
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

inline PageGeom geom(const pct_cache_shape* sh, const int32_t* table,
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

// Checks the pointers and numbers of an attention call, and its arguments.
inline pct_status attend_args(const pct_cache_shape* shape, float scale,
                              const void* q, int64_t q_row_stride,
                              const void* k_cache, const void* v_cache,
                              const int32_t* block_table,
                              const int32_t* ctx_len, const int32_t* n_nodes,
                              const uint64_t* mask, void* out, float* lse,
                              AttendArgs& a) {
  if (!q || !k_cache || !v_cache || !block_table || !out)
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
  return PCT_OK;
}

}  // namespace pct
