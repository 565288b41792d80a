// k_shared.hip -- attention where requests share prefixes, in two parts: the
// rows of a group over its shared keys, as if they were one request's, and
// each request's rows over its own keys behind them.  Both leave sums
// relative to a reference of each row,
//   O = sum_t 2^(z_t - m) v_t, l = sum_t 2^(z_t - m),
// and the join adds them up: m = max(m_1, m_2 ..), O = sum_i 2^(m_i - m) O_i.
// The shared keys are then read once for a group instead of once for each of
// its requests, and the packed rows fill the row tiles.
#include <type_traits>

#include "k_attend_join.h"

namespace pct {

namespace {

constexpr int kJoinThreads = 256, kInFlight = 8;

// Where a row's sums are: slots of a row tile and the row in it.
struct RowSums {
  const float* o;
  const float2* ml;
  int64_t first, step;  // slots first, first + step ..
  int count, mt, row;
};

__device__ __forceinline__ RowSums row_sums(const AttendWs& ws,
                                            const AttendPlan& p, int64_t tile,
                                            const int4& meta, int row) {
  RowSums r{ws.o, ws.ml, 0, 2, 1, p.mt, row};
  if (meta.y < 0) {
    r.first = 2 * (int64_t)p.n_wg + tile;
  } else {
    // the run that began the row tile, then those that went on with it
    r.first = 2 * (int64_t)meta.x;
    r.count = meta.y - meta.x + 1;
  }
  return r;
}

// Row m of request b's packed rows of head h, elements 4 c ..: adds up what
// the runs of both parts left.
template <bool BF16>
__device__ __forceinline__ void join_row(
    const AttendArgs& a, const AttendPlan& ps, const AttendPlan& po,
    const AttendWs& ws, const AttendWs& wo, const int4& rq, const int2& group,
    int b, int h, int m, int c) {
  const PageGeom& g = a.g;
  JoinSum s{neg_inf(), 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  auto add_slots = [&](auto count, const RowSums& r, int dp, int x0)
      __attribute__((always_inline)) {
    constexpr int IN = decltype(count)::value;
    float2 ml[IN];
    float4 o[IN];
#pragma unroll
    for (int k = 0; k < IN; ++k) {
      // (past the last run: that one again, without weight)
      const int x = min(x0 + k, r.count - 1);
      const int64_t slot =
          r.first + r.step * x + (r.count > 1 && x == 0 ? 1 : 0);
      const int64_t row = slot * r.mt + r.row;
      ml[k] = r.ml[row];
      o[k] = reinterpret_cast<const float4*>(r.o + row * dp)[c];
    }
    float m2 = s.m;
#pragma unroll
    for (int k = 0; k < IN; ++k) m2 = fmaxf(m2, ml[k].x);
    s.scale(m2);
#pragma unroll
    for (int k = 0; k < IN; ++k)
      if (x0 + k < r.count) s.add(ml[k], o[k]);
  };
  auto add = [&](const RowSums& r, int dp) __attribute__((always_inline)) {
    if (r.count == 1) {
      add_slots(std::integral_constant<int, 1>{}, r, dp, 0);
    } else if (r.count <= 3) {
      add_slots(std::integral_constant<int, 3>{}, r, dp, 0);
    } else {
      for (int x0 = 0; x0 < r.count; x0 += kInFlight)
        add_slots(std::integral_constant<int, kInFlight>{}, r, dp, x0);
    }
  };
  // (both row tiles' notes on their way before either's sums)
  const int rt = m / po.mt;
  const int64_t own = ((int64_t)b * g.Hkv + h) * wo.row_tiles + rt;
  const int4 own_meta = wo.meta[own];
  if (group.x >= 0) {
    const int pm = rq.w * a.G + m, prt = pm / ps.mt;
    const int64_t tile = (int64_t)h * ws.row_tiles +
                         group.y * a.G / ps.mt + group.x + prt;
    add(row_sums(ws, ps, tile, ws.meta[tile], pm - prt * ps.mt), ps.dp);
  }
  add(row_sums(wo, po, own, own_meta, m - rt * po.mt), po.dp);
  const int i = m / a.G;
  const int64_t row =
      ((int64_t)b * (g.N + 1) + i) * a.Hq + h * a.G + (m - i * a.G);
  // nothing seen: zero (a NaN stays one)
  const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * g.D)[c] =
      make_uint2(round_pair<BF16>(s.o.x * inv, s.o.y * inv),
                 round_pair<BF16>(s.o.z * inv, s.o.w * inv));
  if (a.lse && c == 0)
    a.lse[row] = s.l == 0.f ? neg_inf()
                            : (s.m + (__builtin_log2f(s.l) - kLift<BF16>)) *
                                  (float)kLn2;
}

// A workgroup adds up ROWS rows, LR threads each (4 elements a thread).
template <bool BF16, int LR>
__global__ __launch_bounds__(kJoinThreads) void shared_join_kernel(
    AttendArgs a, AttendPlan ps, AttendPlan po, AttendWs ws, AttendWs wo) {
  constexpr int ROWS = kJoinThreads / LR;
  const PageGeom& g = a.g;
  const int b = blockIdx.x / g.Hkv, h = blockIdx.x - b * g.Hkv;
  const int4 rq = a.share.req[b];
  const int2 group = a.share.group_of[b];
  const int M = (rq.y + 1) * a.G, c = threadIdx.x % LR;
  if (4 * c >= g.D) return;
  for (int m = blockIdx.y * ROWS + threadIdx.x / LR; m < M;
       m += gridDim.y * ROWS)
    join_row<BF16>(a, ps, po, ws, wo, rq, group, b, h, m, c);
}

template <bool BF16, int LR>
hipError_t launch_join(const AttendArgs& a, const AttendPlan& ps,
                       const AttendPlan& po, const AttendWs& ws,
                       const AttendWs& wo, hipStream_t s) {
  constexpr int ROWS = kJoinThreads / LR;
  const int64_t y = ((int64_t)(a.g.N + 1) * a.G + ROWS - 1) / ROWS;
  hipLaunchKernelGGL((shared_join_kernel<BF16, LR>),
                     dim3(a.g.batch * a.g.Hkv, (unsigned)(y < 65535 ? y : 65535)),
                     dim3(kJoinThreads), 0, s, a, ps, po, ws, wo);
  return hipGetLastError();
}

struct Part {
  AttendPlan plan;
  int row_tiles;        // of a request, or of all groups
  int64_t tiles;
  size_t o, ml, meta, end;  // bytes
};

Part part_of(const AttendPlan& p, int64_t row_tiles, int64_t tiles, size_t at) {
  Part x{};
  x.plan = p;
  x.row_tiles = (int)row_tiles;
  x.tiles = tiles;
  const size_t rows = ((size_t)2 * p.n_wg + tiles) * p.mt;
  x.o = at;
  x.ml = x.o + rows * p.dp * sizeof(float);
  x.meta = x.ml + rows * sizeof(float2);
  x.end = x.meta + (size_t)tiles * sizeof(int4);
  return x;
}

struct Parts {
  Part shared, own;
};

Parts parts_of(int batch, int N, int64_t cap, int G, int Hkv, int D) {
  const int64_t M = (int64_t)(N + 1) * G, all = batch * M;
  Parts x;
  AttendPlan p = plan_attend(1, all, cap, Hkv, D);
  // (a group has at least two requests)
  int64_t rt = all / p.mt + batch / 2 + 1;
  x.shared = part_of(p, rt, rt * Hkv, 0);
  p = plan_attend(batch, M, cap, Hkv, D);
  if (p.mt == 128 && p.dp <= 128) p.mt = 64;
  rt = (M + p.mt - 1) / p.mt;
  x.own = part_of(p, rt, rt * Hkv * batch, x.shared.end);
  return x;
}

AttendWs workspace_of(const Part& x, char* base) {
  return AttendWs{reinterpret_cast<float*>(base + x.o),
                  reinterpret_cast<float2*>(base + x.ml),
                  reinterpret_cast<int4*>(base + x.meta), x.row_tiles,
                  x.plan.n_wg};
}

}  // namespace

size_t shared_attention_workspace(const pct_cache_shape& sh) {
  return parts_of(sh.batch, sh.N, (int64_t)sh.max_pages * sh.page_size,
                  sh.Hq / sh.Hkv, sh.Hkv, sh.D)
      .own.end;
}

hipError_t launch_shared_attention(const AttendArgs& a, void* workspace,
                                   hipStream_t s) {
  const PageGeom& g = a.g;
  const Parts x = parts_of(g.batch, g.N, (int64_t)g.max_pages << g.shift, a.G,
                           g.Hkv, g.D);
  char* base = static_cast<char*>(workspace);
  AttendParts parts{{a, a},
                    {x.shared.plan, x.own.plan},
                    {workspace_of(x.shared, base), workspace_of(x.own, base)}};
  parts.a[0].mask = nullptr;
  parts.a[0].g.batch = g.batch / 2;  // groups at most
  if (g.batch == 1) parts.p[0].n_wg = parts.ws[0].n_wg = 0;
  const AttendWs &ws = parts.ws[0], &wo = parts.ws[1];
  const int64_t rows = (int64_t)g.batch * (g.N + 1);
  hipError_t e;
  {
    ProfScope prof(PROF_ATTEND, rows, s);
    switch (x.own.plan.dp) {
      case 64: e = launch_parts_d64(parts, s); break;
      case 96: e = launch_parts_d96(parts, s); break;
      case 128: e = launch_parts_d128(parts, s); break;
      case 192: e = launch_parts_d192(parts, s); break;
      default: e = launch_parts_d256(parts, s); break;
    }
  }
  if (e != hipSuccess) return e;
  ProfScope prof(PROF_JOIN, rows, s);
  const AttendPlan &ps = x.shared.plan, &po = x.own.plan;
  if (a.bf16) {
    if (po.dp <= 64) return launch_join<true, 16>(a, ps, po, ws, wo, s);
    if (po.dp <= 128) return launch_join<true, 32>(a, ps, po, ws, wo, s);
    return launch_join<true, 64>(a, ps, po, ws, wo, s);
  }
  if (po.dp <= 64) return launch_join<false, 16>(a, ps, po, ws, wo, s);
  if (po.dp <= 128) return launch_join<false, 32>(a, ps, po, ws, wo, s);
  return launch_join<false, 64>(a, ps, po, ws, wo, s);
}

}  // namespace pct
