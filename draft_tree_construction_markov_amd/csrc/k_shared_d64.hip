// k_shared_d64.hip -- attention in two parts (shared and own keys) for heads
// padded to 64 elements.
#include "k_shared_launch.h"

namespace pct {
hipError_t launch_parts_d64(const AttendParts& x, hipStream_t s) {
  return launch_parts_dp<64>(x, s);
}
}  // namespace pct
