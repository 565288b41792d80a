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
                                             Lds& mem) {
    attend_tiles<C>(a, ws, block, mem.tiles, mem.odd_s);
  }
};
template <int DP, bool BF16, int PART>
struct PartKernel<DP, 16, BF16, PART> {
  using C = RowsCfg<DP, BF16, PART>;
  using Lds = RowsLds<C>;
  static __device__ __forceinline__ void run(const AttendArgs& a,
                                             const AttendWs& ws, int block,
                                             Lds& mem) {
    attend_rows<C>(a, ws, block, mem);
  }
};

// Own keys first: their reads begin at once, and the products over shared keys
// fill the workgroups' places as these become free.  (One token of 128
// requests, two prefixes; 16 x 65 rows; one token of 64; 32 x 8 rows: 207,
// 196, 60, 64 us; shared keys first 220, 191, 68, 69; by turns 245, 303, 64,
// 71; two launches 209, 202, 65, 74.  4 x 6 rows: 13.4, two launches 21.)
template <class X, class Y>
__global__ __launch_bounds__(256, Y::C::OCC) void attend_parts_kernel(
    AttendParts x) {
  __shared__ union {
    typename X::Lds shared;
    typename Y::Lds own;
  } mem;
  const int b = blockIdx.x, n = x.ws[1].n_wg;
  if (b < n)
    Y::run(x.a[1], x.ws[1], b, mem.own);
  else
    X::run(x.a[0], x.ws[0], b - n, mem.shared);
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
    return launch_both<PartKernel<DP, 128, BF16, kSharedKeys>, Own>(x, s);
  }
  using Own = PartKernel<DP, 64, BF16, kOwnKeys>;
  if (x.p[0].mt == 64)
    return launch_both<PartKernel<DP, 64, BF16, kSharedKeys>, Own>(x, s);
  return launch_both<PartKernel<DP, 128, BF16, kSharedKeys>, Own>(x, s);
}

template <int DP>
hipError_t launch_parts_dp(const AttendParts& x, hipStream_t s) {
  return x.a[0].bf16 ? launch_parts_type<DP, true>(x, s)
                     : launch_parts_type<DP, false>(x, s);
}

template <int DP, bool BF16, int PART>
hipError_t launch_part_type(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, hipStream_t s) {
  if (p.n_wg == 0) return hipSuccess;
  using Half = TilesCfg<DP, 64, BF16, PART>;
  using Full = TilesCfg<DP, 128, BF16, PART>;
  if (p.mt == 64)
    hipLaunchKernelGGL((attend_tiles_kernel<Half>), dim3(p.n_wg),
                       dim3(64 * Half::W), 0, s, a, ws);
  else if (p.mt == 128)
    hipLaunchKernelGGL((attend_tiles_kernel<Full>), dim3(p.n_wg),
                       dim3(64 * Full::W), 0, s, a, ws);
  else
    hipLaunchKernelGGL((attend_rows_kernel<RowsCfg<DP, BF16, PART>>),
                       dim3(p.n_wg), dim3(256), 0, s, a, ws);
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
