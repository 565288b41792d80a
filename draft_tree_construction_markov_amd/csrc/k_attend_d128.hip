// k_attend_d128.hip -- tree attention for heads padded to 128 elements.
#include "k_attend_rows.h"
#include "k_attend_tiles.h"
#include "k_attend_launch.h"

namespace pct {
hipError_t launch_attend_d128(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, hipStream_t s) {
  return launch_attend_dp<128>(a, p, ws, s);
}
}  // namespace pct
