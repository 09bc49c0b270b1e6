// The group-scaled linear for groups of 32 weights.
#include "q4moe_linear.h"

namespace q4 {
hipError_t launch_linear32(const LinearParams& p, hipStream_t stream) { return linear_group<1>(p, stream); }
}  // namespace q4
