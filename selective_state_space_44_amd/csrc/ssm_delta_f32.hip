// ssm_delta_f32.hip -- the walks of the gated delta rule on fp32 inputs
// (ssm_delta_walk.h).
#include "ssm_delta_walk.h"

namespace ssm {
hipError_t launch_delta_walk_f32(const DeltaArgs& a, hipStream_t stream) {
  return launch_walk<float>(a, stream);
}
}  // namespace ssm
