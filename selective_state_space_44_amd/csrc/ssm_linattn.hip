// ssm_linattn.hip -- sums that close the backward of the linear attention with
// one decay per head (gfx950): dk and dv over the query heads that share them,
// the decay's gradient over the walks' blocks, in one launch, each in a fixed
// order.  Bound by HBM: every partial is read once (16384 tokens, 40 heads over
// 8, of 128: 141 us for dk and dv, 5.2 TB/s).  The partials are fp32 in memory
// because a block holds the state of one head only; added by atomics they would
// be summed in no fixed order.
#include "ssm_device.h"
#include "ssm_linattn.h"

namespace ssm {
namespace {

// Four channels of a token and key head: the sum over its query heads.
// Tokens that no sequence holds have no partials, and their sums are not written.
template <typename IO>
__device__ __forceinline__ void group_sum(const LinGroupSum& g, const LinSums& a, int64_t block) {
  const int64_t i = (block * 256 + threadIdx.x) * 4;
  if (i >= g.count) return;
  const int64_t tg = i / g.dim;
  if (a.held && (tg < (int64_t)a.held[0] * a.kvheads || tg >= (int64_t)a.held[1] * a.kvheads))
    return;
  const int per = a.per, d = (int)(i - tg * g.dim);
  const float* p = g.in + tg * per * g.dim + d;
  float4 s = *reinterpret_cast<const float4*>(p);
  for (int h = 1; h < per; ++h) {
    const float4 v = *reinterpret_cast<const float4*>(p + (int64_t)h * g.dim);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  IO* out = static_cast<IO*>(g.out) + i;
  io<IO>::store(out, s.x);
  io<IO>::store(out + 1, s.y);
  io<IO>::store(out + 2, s.z);
  io<IO>::store(out + 3, s.w);
}

__device__ __forceinline__ void dg_sum(const LinSums& a, int head) {
  __shared__ float sums[256];
  float s = 0.0f;
  for (int64_t i = threadIdx.x; i < a.parts; i += 256) s += a.dg_part[i * a.heads + head];
  sums[threadIdx.x] = s;
  __syncthreads();
  for (int m = 128; m > 0; m >>= 1) {
    if ((int)threadIdx.x < m) sums[threadIdx.x] += sums[threadIdx.x + m];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.dg[head] = sums[0];
}

// Blocks: dk's, dv's, then one per head for the decay's gradient.
template <typename IO>
__global__ __launch_bounds__(256) void closing_sums_kernel(LinSums a, uint32_t nk, uint32_t nv) {
  const uint32_t b = blockIdx.x;
  if (b < nk)
    group_sum<IO>(a.k, a, b);
  else if (b < nk + nv)
    group_sum<IO>(a.v, a, b - nk);
  else
    dg_sum(a, (int)(b - nk - nv));
}

}  // namespace

hipError_t launch_closing_sums(const LinSums& a, bool io_bf16, hipStream_t stream) {
  const uint32_t nk = (uint32_t)((a.k.count + 1023) / 1024);
  const uint32_t nv = (uint32_t)((a.v.count + 1023) / 1024);
  const dim3 grid(nk + nv + (a.dg ? (uint32_t)a.heads : 0u));
  if (io_bf16)
    hipLaunchKernelGGL(closing_sums_kernel<bf16>, grid, dim3(256), 0, stream, a, nk, nv);
  else
    hipLaunchKernelGGL(closing_sums_kernel<float>, grid, dim3(256), 0, stream, a, nk, nv);
  return hipGetLastError();
}

}  // namespace ssm
