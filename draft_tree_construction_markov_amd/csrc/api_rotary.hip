// api_rotary.hip -- the C-ABI of rotary positions: the table of frequencies
// and the rows' norm and rotation on their way into the cache.
#include <math.h>

#include "api_cache.h"

using namespace pct;

namespace {

pct_status check_rotary(const pct_rotary* r) {
  if (!r) return fail(PCT_ERR_INVALID_ARG, "rotary is NULL");
  if (r->rot < 0 || r->rot > 256 || r->rot % 2 != 0)
    return fail(PCT_ERR_INVALID_ARG, "rot = %d is not an even number up to 256",
                r->rot);
  if (r->layout != PCT_ROTARY_HALF && r->layout != PCT_ROTARY_INTERLEAVED)
    return fail(PCT_ERR_INVALID_ARG, "unknown rotary layout %d", r->layout);
  if (!isfinite((float)r->amplitude))
    return fail(PCT_ERR_INVALID_ARG, "amplitude must be finite in fp32");
  return PCT_OK;
}

// rows of `heads` heads and of D elements; a null pointer has none
pct_status check_rows(const char* name, const void* x, int64_t stride,
                      int heads, int D) {
  if (!x) return PCT_OK;
  if (stride < (int64_t)heads * D || stride % 8 != 0)
    return fail(PCT_ERR_INVALID_ARG,
                "%s: the row stride must be a multiple of 8 and hold a row",
                name);
  if (!aligned16(x))
    return fail(PCT_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  return PCT_OK;
}

// memory of `rows` rows from x on meets that from y on
bool rows_meet(const void* x, int64_t xs, int64_t xrow, const void* y,
               int64_t ys, int64_t yrow, int64_t rows) {
  const uintptr_t p = (uintptr_t)x, q = (uintptr_t)y;
  return x && y && p < q + 2 * (uintptr_t)((rows - 1) * ys + yrow) &&
         q < p + 2 * (uintptr_t)((rows - 1) * xs + xrow);
}

}  // namespace

extern "C" {

pct_status pct_rotary_table(const pct_rotary* r, uint64_t* table) {
  const pct_status st = check_rotary(r);
  if (st != PCT_OK) return st;
  const int kind = r->scaling;
  if (kind < PCT_ROTARY_PLAIN || kind > PCT_ROTARY_BANDS)
    return fail(PCT_ERR_INVALID_ARG, "unknown rotary scaling %d", kind);
  if (!(r->base > 1.0) || !isfinite(r->base))
    return fail(PCT_ERR_INVALID_ARG, "base must be finite and greater than 1");
  if (kind != PCT_ROTARY_PLAIN && (!(r->factor > 0.0) || !isfinite(r->factor)))
    return fail(PCT_ERR_INVALID_ARG, "factor must be positive and finite");
  if (kind == PCT_ROTARY_BASE && r->rot == 2)
    return fail(PCT_ERR_INVALID_ARG, "a scaled base needs rot > 2");
  if ((kind == PCT_ROTARY_RAMP || kind == PCT_ROTARY_BANDS) &&
      (r->original < 1 || !(r->low > 0.0) || !(r->high > r->low) ||
       !isfinite(r->high)))
    return fail(PCT_ERR_INVALID_ARG,
                "ramps need original >= 1 and 0 < low < high");
  if (r->rot > 0 && !table)
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  const long double two_pi = 6.283185307179586476925286766559L;
  const long double rot = r->rot, s = r->factor;
  long double base = r->base;
  if (kind == PCT_ROTARY_BASE) base *= powl(s, rot / (rot - 2));
  // pair that makes x turns over the original length
  const auto pair_of = [&](long double x) {
    return rot / 2 * logl(r->original / (two_pi * x)) / logl(base);
  };
  long double lo = 0, hi = 0;
  if (kind == PCT_ROTARY_RAMP) {
    lo = floorl(pair_of(r->high));
    hi = ceill(pair_of(r->low));
    lo = lo < 0 ? 0 : lo;
    hi = hi > rot - 1 ? rot - 1 : hi;
    hi = hi - lo < 1e-3L ? lo + 1e-3L : hi;
  }
  for (int i = 0; i < r->rot / 2; ++i) {
    long double f = powl(base, -2 * i / rot);  // radians per position
    long double w = 1;                         // share that is not scaled
    if (kind == PCT_ROTARY_LINEAR) w = 0;
    if (kind == PCT_ROTARY_RAMP) w = 1 - (i - lo) / (hi - lo);
    if (kind == PCT_ROTARY_BANDS)
      w = (r->original * f / two_pi - r->low) / (r->high - r->low);
    w = w < 0 ? 0 : w > 1 ? 1 : w;
    if (kind != PCT_ROTARY_PLAIN && kind != PCT_ROTARY_BASE)
      f = f * w + f / s * (1 - w);
    long double t = f / two_pi;
    t -= floorl(t);
    t = roundl(ldexpl(t, 64));
    table[i] = t >= 18446744073709551616.0L ? 0 : (uint64_t)t;
  }
  return PCT_OK;
}

pct_status pct_cache_write_rotary(
    const pct_cache_shape* shape, const pct_rotary* rotary,
    const uint64_t* table, float eps, const float* q_weight,
    const float* k_weight, const void* q, int64_t q_row_stride, const void* k,
    int64_t k_row_stride, const void* v, int64_t v_row_stride,
    const int32_t* pos, const int64_t* slot, void* q_out,
    int64_t q_out_row_stride, void* k_cache, void* v_cache, void* stream) {
  pct_cache_shape sh;
  if (shape) {
    // neither the block table nor, without queries, their heads are read
    sh = *shape;
    sh.max_pages = 1;
    if (!q) sh.Hq = sh.Hkv;
    shape = &sh;
  }
  pct_status st = check_pages(shape);
  if (st != PCT_OK) return st;
  st = check_heads(shape, q != nullptr);
  if (st != PCT_OK) return st;
  st = check_rotary(rotary);
  if (st != PCT_OK) return st;
  const int D = shape->D;
  if (rotary->rot > D)
    return fail(PCT_ERR_INVALID_ARG, "rot = %d exceeds D = %d", rotary->rot, D);
  if (!(eps >= 0.f) || !isfinite(eps))
    return fail(PCT_ERR_INVALID_ARG, "eps must be finite and not negative");
  if ((!q && !k) || !pos || (rotary->rot > 0 && !table) || !q != !q_out ||
      !k != !v || (k && (!slot || !k_cache || !v_cache)))
    return fail(PCT_ERR_INVALID_ARG, "required pointer is NULL");
  const int64_t rows = (int64_t)shape->batch * (shape->N + 1);
  if ((st = check_rows("q", q, q_row_stride, shape->Hq, D)) != PCT_OK ||
      (st = check_rows("k", k, k_row_stride, shape->Hkv, D)) != PCT_OK ||
      (st = check_rows("v", v, v_row_stride, shape->Hkv, D)) != PCT_OK ||
      (st = check_rows("q_out", q_out, q_out_row_stride, shape->Hq, D)) !=
          PCT_OK)
    return st;
  if (k && (!aligned16(k_cache) || !aligned16(v_cache)))
    return fail(PCT_ERR_INVALID_ARG, "caches must be 16-byte aligned");
  const int64_t qr = (int64_t)shape->Hq * D, kr = (int64_t)shape->Hkv * D;
  if (!(q_out == q && q_out_row_stride == q_row_stride) &&
      (rows_meet(q_out, q_out_row_stride, qr, q, q_row_stride, qr, rows) ||
       rows_meet(q_out, q_out_row_stride, qr, k, k_row_stride, kr, rows) ||
       rows_meet(q_out, q_out_row_stride, qr, v, v_row_stride, kr, rows)))
    return fail(PCT_ERR_INVALID_ARG,
                "q_out overlaps q, k or v without being q");
  RotaryArgs a{};
  a.rows = rows;
  a.shift = log2_of(shape->page_size);
  a.n_slots = (int64_t)shape->n_pages << a.shift;
  a.Hq = shape->Hq;
  a.Hkv = shape->Hkv;
  a.D = D;
  a.bf16 = shape->dtype == PCT_BF16;
  a.rot = rotary->rot;
  a.pairs = rotary->layout == PCT_ROTARY_INTERLEAVED;
  a.freq = table;
  a.amp = (float)rotary->amplitude;
  a.eps = eps;
  a.qw = q_weight;
  a.kw = k_weight;
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = q_row_stride;
  a.ks = k_row_stride;
  a.vs = v_row_stride;
  a.os = q_out_row_stride;
  a.pos = pos;
  a.slot = slot;
  a.out = q_out;
  a.kc = k_cache;
  a.vc = v_cache;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  {
    ProfScope ps(PROF_ROTARY, rows, s);
    e = launch_cache_rotary(a, s);
  }
  if (e != hipSuccess) return hip_fail(e, "rotary kernel");
  return PCT_OK;
}

}  // extern "C"
