// k_attend_launch.h -- the kernel of a plan for one padded head size.
#pragma once
#include "k_attend_rows.h"
#include "k_attend_tiles.h"

namespace pct {

template <int DP, bool BF16>
hipError_t launch_attend_type(const AttendArgs& a, const AttendPlan& p,
                              const AttendWs& ws, hipStream_t s) {
  const dim3 grid(p.n_wg), block(256);
  using Half = TilesCfg<DP, 64, BF16>;
  using Full = TilesCfg<DP, 128, BF16>;
  if (p.mt == 64)
    hipLaunchKernelGGL((attend_tiles_kernel<Half>), grid, dim3(64 * Half::W),
                       0, s, a, ws);
  else if (p.mt == 128)
    hipLaunchKernelGGL((attend_tiles_kernel<Full>), grid, dim3(64 * Full::W),
                       0, s, a, ws);
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
