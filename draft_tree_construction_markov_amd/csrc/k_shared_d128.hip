// k_shared_d128.hip -- attention in two parts (shared and own keys) for heads
// padded to 128 elements.
#include "k_attend_launch.h"

namespace pct {
hipError_t launch_share_d128(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, int part, hipStream_t s) {
  return part == kSharedKeys ? launch_attend_dp<128, kSharedKeys>(a, p, ws, s)
                             : launch_attend_dp<128, kOwnKeys>(a, p, ws, s);
}
}  // namespace pct
