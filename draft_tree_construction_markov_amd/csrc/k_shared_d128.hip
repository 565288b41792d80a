// k_shared_d128.hip -- attention in two parts (shared and own keys) for heads
// padded to 128 elements.
#include "k_shared_launch.h"

namespace pct {
hipError_t launch_parts_d128(const AttendParts& x, hipStream_t s) {
  return launch_parts_dp<128>(x, s);
}
}  // namespace pct
