// ssm_norm.h -- internal interface between the C ABI (ssm_delta_abi.cpp) and the
// layer norm's kernels (ssm_norm.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

constexpr int64_t kMaxNormDim = 16384;

struct NormArgs {
  const void* x;        // [rows, dim], rows x_stride elements apart
  const void* dy;       // backward only
  int64_t x_stride, dy_stride;
  const float* w;       // nullable: 1
  const float* b;       // nullable: 0 (forward only)
  void* out;            // forward: y; backward: dx; contiguous
  float* part;          // backward: [norm_bwd_blocks, 2, dim], null without dw and db
  float* dw;            // nullable
  float* db;            // nullable
  int64_t rows;
  int dim;
  float eps;
};
hipError_t launch_norm_fwd(const NormArgs& a, bool io_bf16, hipStream_t stream);
hipError_t launch_norm_bwd(const NormArgs& a, bool io_bf16, hipStream_t stream);
int norm_bwd_blocks(int64_t rows, int dim, bool io_bf16);

}  // namespace ssm
