// k_shared_launch.h -- the launch of attention in two parts for one padded head
// size: one for both, or a launch for each where a wide head has tiles of 128
// rows (which have 8 waves, the others 4).
#pragma once
#include "k_attend_rows.h"
#include "k_attend_tiles.h"

namespace pct {

template <int DP, int MT, bool BF16, int PART>
struct PartKernel {
  using C = TilesCfg<DP, MT, BF16, PART>;
  using Lds = TilesLds<C>;
  static __device__ __forceinline__ void run(const AttendArgs& a,
                                             const AttendWs& ws, int block,
                                             int blocks, Lds& mem) {
    attend_tiles<C>(a, ws, block, blocks, mem.tiles, mem.odd_s);
  }
};
template <int DP, bool BF16, int PART>
struct PartKernel<DP, 16, BF16, PART> {
  using C = RowsCfg<DP, BF16, PART>;
  using Lds = RowsLds<C>;
  static __device__ __forceinline__ void run(const AttendArgs& a,
                                             const AttendWs& ws, int block,
                                             int blocks, Lds& mem) {
    attend_rows<C>(a, ws, block, blocks, mem);
  }
};

// Little work.  Own keys first: their reads begin at once, and the products over
// shared keys fill the workgroups' places as these become free.  (One token of
// 64 requests, 32 x 8 rows, 4 x 6 rows: 60, 64, 13.4 us; shared keys first 68,
// 69, 13.4; by turns 64, 71, 13.2; two launches 65, 74, 21.)
template <class X, class Y>
__global__ __launch_bounds__(256, Y::C::OCC) void attend_parts_kernel(
    AttendParts x) {
  __shared__ union {
    typename X::Lds shared;
    typename Y::Lds own;
  } mem;
  const int b = blockIdx.x, n = x.ws[1].n_wg;
  if (b < n)
    Y::run(x.a[1], x.ws[1], b, n, mem.own);
  else
    X::run(x.a[0], x.ws[0], b - n, x.ws[0].n_wg, mem.shared);
}

// Much work: every workgroup has one run and stays to the end, and the parts
// have as many of them as their work asks for, by the totals of the share
// plan, so that both end together: the own keys' reads and the products over
// shared keys run side by side all the time.  Work in steps of a shared row
// tile (128 rows by 64 keys): 1.5 for a step of 128 own keys of few rows, 0.8 for
// one of 64 rows by 64 keys, and some steps more for a request's beginning, its
// end and its nodes.  Each part has both places of some compute units and one
// place of others.  One token of 128 requests, two prefixes, 209 -> 180 us (1.2
// in 1.5's place 187, 2.1 217), 16 x 65 rows 197 -> 181, 16 x 16 rows over 16 k
// 99 -> 89; 8 x 257 rows over 8 k, where the shared part alone fills the chip,
// 344 -> 347 (of one state; tree attention of such rows is as fast, with 400 ..
// 600 own keys 374 us and 377).
template <class X, class Y>
__global__ __launch_bounds__(256, 2) void attend_split_kernel(AttendParts x) {
  __shared__ union {
    typename X::Lds shared;
    typename Y::Lds own;
  } mem;
  const AttendArgs& a = x.a[1];
  const float heads = (float)a.g.Hkv, G = (float)a.G;
  const float* t = a.share.totals;
  const float own = t[0], requests = t[1], both = t[2];
  const float shared_cost = heads * G * both * (1.f / (128 * 64));
  float own_cost;
  if constexpr (Y::C::MT == 16) {
    own_cost = 1.5f * heads * (own * (1.f / 128) + 1.5f * requests);
  } else {
    const float tiles = (float)(((a.g.N + 1) * a.G + 63) / 64);
    const float more = 4.f + fmaxf((float)a.g.N * (1.f / 64), 1.f);
    own_cost = 0.8f * heads * tiles * (own * (1.f / 64) + more * requests);
  }
  // places of an XCD (a multiple of 8 workgroups go round the 8 XCDs) that
  // the shared part has
  const int places = gridDim.x >> 3, xcd = blockIdx.x & 7;
  const int at = blockIdx.x >> 3, h = places / 2;
  int n = (int)(places * shared_cost / fmaxf(shared_cost + own_cost, 1.f) +
                0.5f);
  n = both > 0.f ? max(n, 1) : 0;
  n = own > 0.f ? min(n, places - 1) : n;
  n = max(min(n, x.ws[0].n_wg >> 3), places - (x.ws[1].n_wg >> 3));
  // half of them among the first places of the compute units, half among the
  // second ones
  const int n0 = min((n + 1) / 2, h), n1 = n - n0, k = at < h ? at : at - h;
  const bool shared = k < (at < h ? n0 : n1);
  if (shared)
    X::run(x.a[0], x.ws[0], 8 * (at < h ? k : n0 + k) + xcd, 8 * n,
           mem.shared);
  else
    Y::run(x.a[1], x.ws[1], 8 * (at < h ? k - n0 : h - n0 + k - n1) + xcd,
           8 * (places - n), mem.own);
}

// (shared row tiles of 128 rows: so much work that every place has a run)
template <class X, class Y>
hipError_t launch_split(const AttendParts& x, hipStream_t s) {
  const int n = x.ws[0].n_wg > x.ws[1].n_wg ? x.ws[0].n_wg : x.ws[1].n_wg;
  hipLaunchKernelGGL((attend_split_kernel<X, Y>), dim3(n), dim3(256), 0, s, x);
  return hipGetLastError();
}

template <class X, class Y>
hipError_t launch_both(const AttendParts& x, hipStream_t s) {
  hipLaunchKernelGGL((attend_parts_kernel<X, Y>),
                     dim3(x.ws[0].n_wg + x.ws[1].n_wg), dim3(256), 0, s, x);
  return hipGetLastError();
}

// Own keys have row tiles of 16 or 64 rows, shared ones of as many or more.
template <int DP, bool BF16>
hipError_t launch_parts_type(const AttendParts& x, hipStream_t s) {
  if (x.p[1].mt == 16) {
    using Own = PartKernel<DP, 16, BF16, kOwnKeys>;
    if (x.p[0].mt == 16)
      return launch_both<PartKernel<DP, 16, BF16, kSharedKeys>, Own>(x, s);
    if (x.p[0].mt == 64)
      return launch_both<PartKernel<DP, 64, BF16, kSharedKeys>, Own>(x, s);
    return launch_split<PartKernel<DP, 128, BF16, kSharedKeys>, Own>(x, s);
  }
  using Own = PartKernel<DP, 64, BF16, kOwnKeys>;
  if (x.p[0].mt == 64)
    return launch_both<PartKernel<DP, 64, BF16, kSharedKeys>, Own>(x, s);
  return launch_split<PartKernel<DP, 128, BF16, kSharedKeys>, Own>(x, s);
}

template <int DP>
hipError_t launch_parts_dp(const AttendParts& x, hipStream_t s) {
  return x.a[0].bf16 ? launch_parts_type<DP, true>(x, s)
                     : launch_parts_type<DP, false>(x, s);
}

// One part of wide heads.  (Shared keys come here with tiles of 128 rows only.)
template <int DP, bool BF16, int PART>
hipError_t launch_part_type(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, hipStream_t s) {
  if (p.n_wg == 0) return hipSuccess;
  using Full = TilesCfg<DP, 128, BF16, PART>;
  if constexpr (PART == kOwnKeys) {
    using Half = TilesCfg<DP, 64, BF16, PART>;
    using Rows = RowsCfg<DP, BF16, PART>;
    if (p.mt == 64)
      hipLaunchKernelGGL((attend_tiles_kernel<Half>), dim3(p.n_wg),
                         dim3(64 * Half::W), 0, s, a, ws);
    if (p.mt == 16)
      hipLaunchKernelGGL((attend_rows_kernel<Rows>), dim3(p.n_wg), dim3(256),
                         0, s, a, ws);
    if (p.mt < 128) return hipGetLastError();
  }
  hipLaunchKernelGGL((attend_tiles_kernel<Full>), dim3(p.n_wg),
                     dim3(64 * Full::W), 0, s, a, ws);
  return hipGetLastError();
}

// Wide heads: one launch unless there are row tiles of 128 rows.
template <int DP, bool BF16>
hipError_t launch_parts_small(const AttendParts& x, hipStream_t s) {
  using Rows = PartKernel<DP, 16, BF16, kOwnKeys>;
  using Tiles = PartKernel<DP, 64, BF16, kOwnKeys>;
  using Shared = PartKernel<DP, 64, BF16, kSharedKeys>;
  if (x.p[1].mt > 16) return launch_both<Shared, Tiles>(x, s);
  if (x.p[0].mt > 16) return launch_both<Shared, Rows>(x, s);
  return launch_both<PartKernel<DP, 16, BF16, kSharedKeys>, Rows>(x, s);
}
template <int DP>
hipError_t launch_parts_wide(const AttendParts& x, hipStream_t s) {
  if (x.p[0].mt <= 64 && x.p[1].mt <= 64)
    return x.a[0].bf16 ? launch_parts_small<DP, true>(x, s)
                       : launch_parts_small<DP, false>(x, s);
  hipError_t e =
      x.a[0].bf16
          ? launch_part_type<DP, true, kSharedKeys>(x.a[0], x.p[0], x.ws[0], s)
          : launch_part_type<DP, false, kSharedKeys>(x.a[0], x.p[0], x.ws[0],
                                                     s);
  if (e != hipSuccess) return e;
  return x.a[1].bf16
             ? launch_part_type<DP, true, kOwnKeys>(x.a[1], x.p[1], x.ws[1], s)
             : launch_part_type<DP, false, kOwnKeys>(x.a[1], x.p[1], x.ws[1],
                                                     s);
}

}  // namespace pct
