// k_shared_d192.hip -- attention in two parts (shared and own keys) for heads
// padded to 192 elements.
#include "k_shared_launch.h"

namespace pct {
hipError_t launch_parts_d192(const AttendParts& x, hipStream_t s) {
  return launch_parts_wide<192>(x, s);
}
}  // namespace pct
