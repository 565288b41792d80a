// k_shared_d96.hip -- attention in two parts (shared and own keys) for heads
// padded to 96 elements.
#include "k_shared_launch.h"

namespace pct {
hipError_t launch_parts_d96(const AttendParts& x, hipStream_t s) {
  return launch_parts_dp<96>(x, s);
}
}  // namespace pct
