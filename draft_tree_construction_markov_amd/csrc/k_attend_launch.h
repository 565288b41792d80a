// k_attend_launch.h -- the kernel of a plan for one padded head size.
#pragma once
#include "k_attend_rows.h"
#include "k_attend_tiles.h"

namespace pct {

template <int DP, bool BF16>
hipError_t launch_attend_type(const AttendArgs& a, const AttendPlan& p,
                              const AttendWs& ws, hipStream_t s) {
  const dim3 grid(p.n_wg), block(256);
  if (p.shared && p.nt == 1)
    hipLaunchKernelGGL((attend_tiles_kernel<TilesCfg<DP, 1, BF16>>), grid,
                       block, 0, s, a, ws);
  else if (p.shared)
    hipLaunchKernelGGL((attend_tiles_kernel<TilesCfg<DP, 2, BF16>>), grid,
                       block, 0, s, a, ws);
  else
    hipLaunchKernelGGL((attend_rows_kernel<RowsCfg<DP, BF16>>), grid, block,
                       0, s, a, ws);
  return hipGetLastError();
}

template <int DP>
hipError_t launch_attend_dp(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, hipStream_t s) {
  return a.bf16 ? launch_attend_type<DP, true>(a, p, ws, s)
                : launch_attend_type<DP, false>(a, p, ws, s);
}

}  // namespace pct
