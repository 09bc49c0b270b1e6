// The group-scaled linear: dispatch by group size.
#include "q4moe_linear.h"

namespace q4 {

hipError_t launch_linear(const LinearParams& p, hipStream_t stream) {
  if (p.group == 32) return launch_linear32(p, stream);
  if (p.group == 64) return launch_linear64(p, stream);
  return launch_linear128(p, stream);
}

}  // namespace q4
