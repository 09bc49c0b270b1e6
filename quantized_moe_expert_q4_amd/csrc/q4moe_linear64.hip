// The group-scaled linear for groups of 64 weights.
#include "q4moe_linear.h"

namespace q4 {
hipError_t launch_linear64(const LinearParams& p, hipStream_t stream) { return linear_group<2>(p, stream); }
}  // namespace q4
