// ssm_linattn.hip -- sums that close the backward of the linear attention with
// one decay per head (gfx950): dk and dv over the query heads that share them,
// the decay's gradient over the walks' blocks.  Each in a fixed order.  Bound by
// HBM: every partial is read once (16384 tokens, 40 heads over 8, of 128: 73 us
// for each of dk and dv, 5.0 TB/s).  The partials are fp32 in memory because a
// block holds the state of one head only; added by atomics they would be summed
// in no fixed order.
#include "ssm_device.h"
#include "ssm_linattn.h"

namespace ssm {
namespace {

template <typename IO>
__global__ __launch_bounds__(256) void group_sum_kernel(const float* in, IO* out, int64_t n,
                                                        int per, int dim) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const int64_t tg = i / dim;
  const int d = (int)(i - tg * dim);
  const float* p = in + tg * per * dim + d;
  float4 s = *reinterpret_cast<const float4*>(p);
  for (int h = 1; h < per; ++h) {
    const float4 v = *reinterpret_cast<const float4*>(p + (int64_t)h * dim);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  io<IO>::store(out + i, s.x);
  io<IO>::store(out + i + 1, s.y);
  io<IO>::store(out + i + 2, s.z);
  io<IO>::store(out + i + 3, s.w);
}

__global__ __launch_bounds__(256) void dg_sum_kernel(const float* part, float* dg, int64_t parts,
                                                     int heads) {
  __shared__ float sums[256];
  float s = 0.0f;
  for (int64_t i = threadIdx.x; i < parts; i += 256) s += part[i * heads + blockIdx.x];
  sums[threadIdx.x] = s;
  __syncthreads();
  for (int m = 128; m > 0; m >>= 1) {
    if ((int)threadIdx.x < m) sums[threadIdx.x] += sums[threadIdx.x + m];
    __syncthreads();
  }
  if (threadIdx.x == 0) dg[blockIdx.x] = sums[0];
}

}  // namespace

hipError_t launch_dg_sum(const float* part, float* dg, int64_t parts, int heads,
                         hipStream_t stream) {
  hipLaunchKernelGGL(dg_sum_kernel, dim3(heads), dim3(256), 0, stream, part, dg, parts, heads);
  return hipGetLastError();
}

hipError_t launch_group_sum(const float* in, void* out, int64_t tokens, int groups, int per,
                            int dim, bool io_bf16, hipStream_t stream) {
  const int64_t n = tokens * groups * dim;
  const dim3 grid((unsigned)((n / 4 + 255) / 256));
  if (io_bf16)
    hipLaunchKernelGGL(group_sum_kernel<bf16>, grid, dim3(256), 0, stream, in,
                       static_cast<bf16*>(out), n, per, dim);
  else
    hipLaunchKernelGGL(group_sum_kernel<float>, grid, dim3(256), 0, stream, in,
                       static_cast<float*>(out), n, per, dim);
  return hipGetLastError();
}

}  // namespace ssm
