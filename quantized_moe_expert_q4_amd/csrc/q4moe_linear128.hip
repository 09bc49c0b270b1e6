// The group-scaled linear for groups of 128 weights.
#include "q4moe_linear.h"

namespace q4 {
hipError_t launch_linear128(const LinearParams& p, hipStream_t stream) { return linear_group<4>(p, stream); }
}  // namespace q4
