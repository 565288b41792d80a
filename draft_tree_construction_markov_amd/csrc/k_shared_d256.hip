// k_shared_d256.hip -- attention in two parts (shared and own keys) for heads
// padded to 256 elements.
#include "k_shared_launch.h"

namespace pct {
hipError_t launch_parts_d256(const AttendParts& x, hipStream_t s) {
  return launch_parts_wide<256>(x, s);
}
}  // namespace pct
