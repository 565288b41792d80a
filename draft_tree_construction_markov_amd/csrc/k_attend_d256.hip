// k_attend_d256.hip -- tree attention for heads padded to 256 elements.
#include "k_attend_rows.h"
#include "k_attend_tiles.h"
#include "k_attend_launch.h"

namespace pct {
hipError_t launch_attend_d256(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, hipStream_t s) {
  return launch_attend_dp<256>(a, p, ws, s);
}
}  // namespace pct
