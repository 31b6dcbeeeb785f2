// ssm_delta_mm.hip -- the walks of the gated delta rule on bf16 inputs
// (ssm_delta_walk.h).
#include "ssm_delta_walk.h"

namespace ssm {
hipError_t launch_delta_walk_mm(const DeltaArgs& a, hipStream_t stream) {
  return launch_walk<bf16>(a, stream);
}
}  // namespace ssm
