// k_shared_d64.hip -- attention in two parts (shared and own keys) for heads
// padded to 64 elements.
#include "k_attend_launch.h"

namespace pct {
hipError_t launch_share_d64(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, int part, hipStream_t s) {
  return part == kSharedKeys ? launch_attend_dp<64, kSharedKeys>(a, p, ws, s)
                             : launch_attend_dp<64, kOwnKeys>(a, p, ws, s);
}
}  // namespace pct
