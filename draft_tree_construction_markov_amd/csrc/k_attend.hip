// k_attend.hip -- tree attention: the choice of tile, the workspace and the
// join of row tiles whose keys were split over workgroups.
#include <type_traits>

#include "k_attend_join.h"

namespace pct {

namespace {

int padded(int D) {
  return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : D <= 192 ? 192 : 256;
}

}  // namespace

// rows: packed rows of a request and key-value head, at most
AttendPlan plan_attend(int requests, int64_t rows, int64_t cap, int Hkv,
                       int D) {
  const int64_t batch = requests, M = rows;
  AttendPlan p{};
  p.dp = padded(D);
  // The smallest row tile that holds a request's rows of one head, or 64 rows
  // for little work; waves with keys of their own up to 16 rows (with 32, 64
  // requests of 8 rows over up to 8 k positions took 205 us, with shared
  // tiles 166).
  p.mt = M <= 16 ? 16 : M <= 64 ? 64 : 128;
  // (bounded, so that no shape overflows the products below)
  const auto bounded = [](int64_t x) { return x < 1 << 30 ? x : 1 << 30; };
  const int64_t key_tiles = (cap + kTilesKb - 1) / kTilesKb;
  if (p.mt == 128 && p.dp <= 128 &&
      bounded(batch * (Hkv * ((M + 127) / 128))) * key_tiles <= kHalfUnits)
    p.mt = 64;
  const bool shared = p.mt > 16;
  p.ks = shared ? kTilesKb : 4 * kRowsKb;
  // as many runs as stay on the chip, or as the longest requests could fill
  const int64_t steps = (cap + p.ks - 1) / p.ks;
  const int64_t row_tiles = (M + p.mt - 1) / p.mt;
  const int64_t tiles = batch * (Hkv * row_tiles);
  const int64_t units = bounded(tiles) * steps;
  const int few = shared ? kTilesFew : kRowsFew;
  const int64_t runs = units / (steps < few ? steps : few) + 1;
  p.n_wg = kCus * (p.dp <= 128 ? 2 : 1);
  if (runs < p.n_wg) p.n_wg = (int)(runs + 7) / 8 * 8;
  if (tiles <= p.n_wg) {
    p.row_tiles = (int)row_tiles;
    p.tiles = (int)tiles;
  }
  p.groups = p.mt <= 16 || p.n_wg >= 16 * tiles ? 4 : 1;
  return p;
}

namespace {

struct WsLayout {
  size_t o, ml, meta, total;
};

WsLayout layout(const AttendPlan& p) {
  WsLayout w{};
  const size_t rows = (size_t)2 * p.n_wg * p.mt;
  w.o = 0;
  w.ml = rows * p.dp * sizeof(float);
  w.meta = w.ml + rows * sizeof(float2);
  w.total = w.meta + (size_t)p.n_wg * sizeof(int4);
  return w;
}

}  // namespace

// A workgroup adds up ROWS rows of a row tile that starts in one run and ends
// in a later one: LR threads per row (4 elements each), PG groups of
// runs side by side, kInFlight runs of a group loaded at a time:
//   m = max_w m_w, out = sum_w 2^(m_w - m) O_w / sum_w 2^(m_w - m) l_w,
// in order of runs within a group, then of groups.  PG = 4 where rows are few
// or split over many runs (32 rows over 60 k positions: 56 us with the
// attention, 66 with one group), else one (512 rows over up to 5 k: 87 us,
// 96 with four).  A workgroup for every row tile if these are fewer than the
// runs, else for every run; the others leave at once, but 8192 of them took
// 3 us.  Bound by the sums' read: 32 trees of 257 rows 16 us for 66 MB.
constexpr int kJoinThreads = 256, kInFlight = 8;

template <bool BF16, int LR, int PG>
__global__ __launch_bounds__(kJoinThreads) void attend_join_kernel(
    AttendArgs a, AttendPlan p, AttendWs ws) {
  constexpr int ROWS = kJoinThreads / LR / PG;
  __shared__ float4 o_s[PG > 1 ? kJoinThreads : 1];
  __shared__ float2 ml_s[PG > 1 ? kJoinThreads : 1];
  const PageGeom& g = a.g;
  const int4 seg = ws.meta[blockIdx.x];
  int b = seg.x, h = seg.y >> 20, rt = seg.y & 0xfffff;
  if (p.row_tiles > 0) {
    // entries of row tiles that the request does not have are not written
    h = blockIdx.x / p.row_tiles;
    rt = blockIdx.x - h * p.row_tiles;
    b = h / g.Hkv;
    h -= b * g.Hkv;
  } else if (seg.w < 0) {
    return;
  }
  const int n = g.n_nodes ? clamp_nodes(g.n_nodes[b], g.N) : g.N;
  if (rt * p.mt >= (n + 1) * a.G || seg.w < 0) return;
  const int run = seg.z, runs = seg.w - run + 1;
  const int tid = threadIdx.x;
  const int c = tid % LR, pg = tid / (LR * ROWS);
  const int r = blockIdx.y * ROWS + tid / LR % ROWS;
  const int m = rt * p.mt + r;
  const bool live = m < (n + 1) * a.G && 4 * c < g.D;
  JoinSum s{neg_inf(), 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  auto add_runs = [&](auto count, int x0) __attribute__((always_inline)) {
    constexpr int IN = decltype(count)::value;
    float2 ml[IN];
    float4 o[IN];
#pragma unroll
    for (int k = 0; k < IN; ++k) {
      // (past the last run: that one again, without weight)
      const int x = min(x0 + k * PG, runs - 1);
      const int64_t row =
          (int64_t)(2 * (run + x) + (x == 0 ? 1 : 0)) * p.mt + r;
      ml[k] = ws.ml[row];
      o[k] = reinterpret_cast<const float4*>(ws.o + row * p.dp)[c];
    }
    float m2 = s.m;
#pragma unroll
    for (int k = 0; k < IN; ++k) m2 = fmaxf(m2, ml[k].x);
    s.scale(m2);
#pragma unroll
    for (int k = 0; k < IN; ++k)
      if (x0 + k * PG < runs) s.add(ml[k], o[k]);
  };
  if (live) {
    if (runs <= 2 * PG) {
      if (pg < runs) add_runs(std::integral_constant<int, 2>{}, pg);
    } else {
      for (int x0 = pg; x0 < runs; x0 += kInFlight * PG)
        add_runs(std::integral_constant<int, kInFlight>{}, x0);
    }
  }
  if constexpr (PG > 1) {
    o_s[tid] = s.o;
    ml_s[tid] = make_float2(s.m, s.l);
    __syncthreads();
    if (pg > 0) return;
    float m2 = s.m;
#pragma unroll
    for (int y = 1; y < PG; ++y) m2 = fmaxf(m2, ml_s[tid + y * LR * ROWS].x);
    s.scale(m2);
#pragma unroll
    for (int y = 1; y < PG; ++y)
      s.add(ml_s[tid + y * LR * ROWS], o_s[tid + y * LR * ROWS]);
  }
  if (!live) return;
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

template <bool BF16, int LR>
hipError_t launch_join(const AttendArgs& a, const AttendPlan& p,
                       const AttendWs& ws, hipStream_t s) {
  const int x = p.row_tiles > 0 ? p.tiles : p.n_wg;
  if (p.groups > 1)
    hipLaunchKernelGGL((attend_join_kernel<BF16, LR, 4>),
                       dim3(x, p.mt / (kJoinThreads / LR / 4)),
                       dim3(kJoinThreads), 0, s, a, p, ws);
  else
    hipLaunchKernelGGL((attend_join_kernel<BF16, LR, 1>),
                       dim3(x, p.mt / (kJoinThreads / LR)),
                       dim3(kJoinThreads), 0, s, a, p, ws);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_join_type(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, hipStream_t s) {
  if (p.dp <= 64) return launch_join<BF16, 16>(a, p, ws, s);
  if (p.dp <= 128) return launch_join<BF16, 32>(a, p, ws, s);
  return launch_join<BF16, 64>(a, p, ws, s);
}

size_t tree_attention_workspace(const pct_cache_shape& sh) {
  return layout(plan_attend(sh.batch, (int64_t)(sh.N + 1) * (sh.Hq / sh.Hkv),
                            (int64_t)sh.max_pages * sh.page_size, sh.Hkv,
                            sh.D))
      .total;
}

hipError_t launch_tree_attention(const AttendArgs& a, void* workspace,
                                 hipStream_t s) {
  const PageGeom& g = a.g;
  const AttendPlan p =
      plan_attend(g.batch, (int64_t)(g.N + 1) * a.G,
                  (int64_t)g.max_pages << g.shift, g.Hkv, g.D);
  const WsLayout w = layout(p);
  char* base = static_cast<char*>(workspace);
  AttendWs ws{reinterpret_cast<float*>(base + w.o),
              reinterpret_cast<float2*>(base + w.ml),
              reinterpret_cast<int4*>(base + w.meta), p.row_tiles, p.n_wg};
  hipError_t e;
  {
    ProfScope ps(PROF_ATTEND, (int64_t)g.batch * (g.N + 1), s);
    switch (p.dp) {
      case 64: e = launch_attend_d64(a, p, ws, s); break;
      case 96: e = launch_attend_d96(a, p, ws, s); break;
      case 128: e = launch_attend_d128(a, p, ws, s); break;
      case 192: e = launch_attend_d192(a, p, ws, s); break;
      default: e = launch_attend_d256(a, p, ws, s); break;
    }
  }
  if (e != hipSuccess) return e;
  ProfScope ps(PROF_JOIN, (int64_t)g.batch * (g.N + 1), s);
  return a.bf16 ? launch_join_type<true>(a, p, ws, s)
                : launch_join_type<false>(a, p, ws, s);
}

}  // namespace pct
