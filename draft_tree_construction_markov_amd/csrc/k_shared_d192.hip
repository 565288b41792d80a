// k_shared_d192.hip -- attention in two parts (shared and own keys) for heads
// padded to 192 elements.
#include "k_attend_launch.h"

namespace pct {
hipError_t launch_share_d192(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, int part, hipStream_t s) {
  return part == kSharedKeys ? launch_attend_dp<192, kSharedKeys>(a, p, ws, s)
                             : launch_attend_dp<192, kOwnKeys>(a, p, ws, s);
}
}  // namespace pct
