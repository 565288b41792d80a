// k_shared.hip -- attention where requests share prefixes, in two parts: the
// rows of a group over its shared keys, as if they were one request's, and
// each request's rows over its own keys behind them.  Both leave sums
// relative to a reference of each row,
//   O = sum_t 2^(z_t - m) v_t, l = sum_t 2^(z_t - m),
// and the join adds them up: m = max(m_1, m_2 ..), O = sum_i 2^(m_i - m) O_i.
// The shared keys are then read once for a group instead of once for each of
// its requests, and the packed rows fill the row tiles.  On the same inputs
// again and again, one token of 128 requests over two prefixes of 16 k
// positions and 64 .. 4096 own ones 176 us (tree attention 1259), 16 requests
// of 65 rows over 8 k 185 (242), 790 TFLOP/s.  The join is bound by the sums'
// read: 6 and 16 us of these.  All rows leave sums, those of requests without
// a group too: 32 x 257 rows over 1 k .. 4 k positions 811 us (495), over a
// shared 8 k 1476 (1391).
#include "k_attend_join.h"

namespace pct {

namespace {

constexpr int kJoinThreads = 256, kInFlight = 8;
// Up to so many tiles of 128 rows by 64 keys, if requests are as long as the
// block table allows, wide heads have tiles of 64 rows, which go into one
// launch with the own keys: D = 256, 8 x 4 rows over 2 k shared positions (140
// tiles) 38 -> 25 us, one token of 64 requests over 4 k (1104) 62 -> 57, but 64
// x 4 rows over 4 k, D = 192 (4416) 77 -> 90, 16 x 65 rows over 8 k (18 k) 224
// -> 326.
constexpr int kOneLaunch = 2048;

// Where a row's sums are: slots of a row tile and the row in it.
struct RowSums {
  const float* o;
  const float2* ml;
  int64_t first;  // slots first, first + 2 ..
  int count, mt, row;
};

__device__ __forceinline__ RowSums row_sums(const AttendWs& ws,
                                            const AttendPlan& p, int64_t tile,
                                            const int4& meta, int row) {
  RowSums r{ws.o, ws.ml, 0, 1, p.mt, row};
  if (meta.y < 0) {
    r.first = 2 * (int64_t)p.n_wg + tile;
  } else {
    // the run that began the row tile, then those that went on with it
    r.first = 2 * (int64_t)meta.x;
    r.count = meta.y - meta.x + 1;
  }
  return r;
}

// Adds the sums x0, x0 + STEP .. (IN of them) of a row, elements 4 c .. .
template <int IN, int STEP>
__device__ __forceinline__ void add_slots(JoinSum& s, const RowSums& r, int dp,
                                          int c, int x0) {
  float2 ml[IN];
  float4 o[IN];
#pragma unroll
  for (int k = 0; k < IN; ++k) {
    // (past the last run: that one again, without weight)
    const int x = min(x0 + k * STEP, r.count - 1);
    const int64_t slot = r.first + 2 * x + (r.count > 1 && x == 0 ? 1 : 0);
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
    if (x0 + k * STEP < r.count) s.add(ml[k], o[k]);
}

// The sums that group pg of PG has of a row: in few loads where they are few.
template <int PG>
__device__ __forceinline__ void add_sums(JoinSum& s, const RowSums& r, int dp,
                                         int c, int pg) {
  if (pg >= r.count) return;
  if (r.count <= PG) {
    add_slots<1, PG>(s, r, dp, c, pg);
  } else if (r.count <= 3 * PG) {
    add_slots<3, PG>(s, r, dp, c, pg);
  } else {
    for (int x0 = pg; x0 < r.count; x0 += kInFlight * PG)
      add_slots<kInFlight, PG>(s, r, dp, c, x0);
  }
}

// A workgroup adds up ROWS rows of a request and head, LR threads each (4
// elements a thread), PG groups of runs side by side: in the order of the
// runs within a group, then of the groups.
template <bool BF16, int LR, int PG>
__global__ __launch_bounds__(kJoinThreads) void shared_join_kernel(
    AttendArgs a, AttendPlan ps, AttendPlan po, AttendWs ws, AttendWs wo) {
  constexpr int ROWS = kJoinThreads / LR / PG;
  __shared__ float4 o_s[PG > 1 ? kJoinThreads : 1];
  __shared__ float2 ml_s[PG > 1 ? kJoinThreads : 1];
  const PageGeom& g = a.g;
  const int b = blockIdx.x / g.Hkv, h = blockIdx.x - b * g.Hkv;
  const int4 rq = a.share.req[b];
  const int2 group = a.share.group_of[b];
  const int tid = threadIdx.x, M = (rq.y + 1) * a.G;
  const int c = tid % LR, pg = tid / (LR * ROWS);
  for (int m0 = blockIdx.y * ROWS; m0 < M; m0 += gridDim.y * ROWS) {
    const int m = m0 + tid / LR % ROWS;
    const bool live = m < M && 4 * c < g.D;
    JoinSum s{neg_inf(), 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (live) {
      // (both row tiles' notes on their way before either's sums)
      const int rt = m / po.mt;
      const int64_t own = ((int64_t)b * g.Hkv + h) * wo.row_tiles + rt;
      const int4 own_meta = wo.meta[own];
      if (group.x >= 0) {
        const int pm = rq.w * a.G + m, prt = pm / ps.mt;
        const int64_t tile = (int64_t)h * ws.row_tiles +
                             group.y * a.G / ps.mt + group.x + prt;
        add_sums<PG>(s,
                     row_sums(ws, ps, tile, ws.meta[tile], pm - prt * ps.mt),
                     ps.dp, c, pg);
      }
      // (from the last group on, which has the fewest of the others)
      add_sums<PG>(s, row_sums(wo, po, own, own_meta, m - rt * po.mt), po.dp,
                   c, PG - 1 - pg);
    }
    if constexpr (PG > 1) {
      __syncthreads();  // the previous row's are read
      o_s[tid] = s.o;
      ml_s[tid] = make_float2(s.m, s.l);
      __syncthreads();
      if (pg > 0) continue;
      float m2 = s.m;
#pragma unroll
      for (int y = 1; y < PG; ++y) m2 = fmaxf(m2, ml_s[tid + y * LR * ROWS].x);
      s.scale(m2);
#pragma unroll
      for (int y = 1; y < PG; ++y)
        s.add(ml_s[tid + y * LR * ROWS], o_s[tid + y * LR * ROWS]);
    }
    if (!live) continue;
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
}

template <bool BF16, int LR, int PG>
hipError_t launch_join_groups(const AttendArgs& a, const AttendParts& x,
                              hipStream_t s) {
  constexpr int ROWS = kJoinThreads / LR / PG;
  const int64_t y = ((int64_t)(a.g.N + 1) * a.G + ROWS - 1) / ROWS;
  hipLaunchKernelGGL((shared_join_kernel<BF16, LR, PG>),
                     dim3(a.g.batch * a.g.Hkv,
                          (unsigned)(y < 65535 ? y : 65535)),
                     dim3(kJoinThreads), 0, s, a, x.p[0], x.p[1], x.ws[0],
                     x.ws[1]);
  return hipGetLastError();
}

template <bool BF16, int LR>
hipError_t launch_join(const AttendArgs& a, const AttendParts& x, int groups,
                       hipStream_t s) {
  return groups > 1 ? launch_join_groups<BF16, LR, 4>(a, x, s)
                    : launch_join_groups<BF16, LR, 1>(a, x, s);
}

template <bool BF16>
hipError_t launch_join_type(const AttendArgs& a, const AttendParts& x,
                            int groups, hipStream_t s) {
  if (x.p[1].dp <= 64) return launch_join<BF16, 16>(a, x, groups, s);
  if (x.p[1].dp <= 128) return launch_join<BF16, 32>(a, x, groups, s);
  return launch_join<BF16, 64>(a, x, groups, s);
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
  const int64_t steps = (cap + kTilesKb - 1) / kTilesKb;
  const bool one = p.dp > 128 && steps * ((all + 127) / 128) * Hkv <= kOneLaunch;
  if (one && p.mt == 128) p.mt = 64;
  // (a group has at least two requests)
  int64_t rt = all / p.mt + batch / 2 + 1;
  x.shared = part_of(p, rt, rt * Hkv, 0);
  p = plan_attend(batch, M, cap, Hkv, D);
  if (p.mt == 128 && (p.dp <= 128 || one)) p.mt = 64;
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
  // Groups where the shared row tiles are cut into many runs each (7 tokens
  // over 31 k shared positions, 2 heads, 256 runs: 53 us without, 30 with; 123
  // tokens over 16 k, 8 heads, 512 runs of 40 row tiles: 209 and 211).
  const int64_t tiles =
      ((int64_t)g.batch * (g.N + 1) * a.G / x.shared.plan.mt + 1) * g.Hkv;
  const int groups = x.shared.plan.n_wg >= 16 * tiles ? 4 : 1;
  return a.bf16 ? launch_join_type<true>(a, parts, groups, s)
                : launch_join_type<false>(a, parts, groups, s);
}

}  // namespace pct
