// k_attend_d192.hip -- tree attention for heads padded to 192 elements.
#include "k_attend_rows.h"
#include "k_attend_tiles.h"
#include "k_attend_launch.h"

namespace pct {
hipError_t launch_attend_d192(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, hipStream_t s) {
  return launch_attend_dp<192>(a, p, ws, s);
}
}  // namespace pct
