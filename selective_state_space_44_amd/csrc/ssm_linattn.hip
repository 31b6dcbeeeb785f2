// ssm_linattn.hip -- linear attention with one decay per head over whole
// sequences (gfx950, wave64): S_t = a S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.
//
// The recurrence as written: eight lanes own a row of S, 32 rows to a block,
// and walk the tokens with the state in registers.
#include "ssm_device.h"
#include "ssm_linattn.h"

namespace ssm {
namespace {

template <typename IO, int E, bool TAN>
__global__ __launch_bounds__(256) void linattn_walk_kernel(LinArgs a, int vblocks) {
  const int c = threadIdx.x & 7;
  const int64_t sh = blockIdx.x / vblocks;
  const int row = (int)(blockIdx.x % vblocks) * 32 + (threadIdx.x >> 3);
  const int64_t seq = sh / a.heads;
  const int head = (int)(sh - seq * a.heads);
  int64_t first = seq * a.seqlen, len = a.seqlen;
  if (a.cu) {
    const int64_t lo = a.cu[seq], hi = a.cu[seq + 1];
    first = lo < 0 ? 0 : lo > a.tokens ? a.tokens : lo;
    const int64_t end = hi < first ? first : hi > a.tokens ? a.tokens : hi;
    len = end - first;
  }
  const bool on = row < a.vd;
  const float g = a.log_decay[head] * kLog2e;
  const float decay = fast_exp2(g);
  float s[E], ds[E];
  float dg = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int d = e * 8 + c;
    s[e] = ds[e] = 0.0f;
    if (a.s0 && on && d < a.kd)
      s[e] = a.s0_swap ? a.s0[(sh * a.kd + d) * a.vd + row] : a.s0[(sh * a.vd + row) * a.kd + d];
  }
  const IO* q = static_cast<const IO*>(a.q.p) + (int64_t)(head / a.q.hdiv) * a.kd;
  const IO* k = static_cast<const IO*>(a.k.p) + (int64_t)(head / a.k.hdiv) * a.kd;
  const IO* v = static_cast<const IO*>(a.v.p) + (int64_t)(head / a.v.hdiv) * a.vd;
  for (int64_t i = 0; i < len; ++i) {
    const int64_t t = a.rev ? first + len - 1 - i : first + i;
    const float vt = on ? io<IO>::load(v + t * a.v.stride + row) : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = e * 8 + c;
      if (d < a.kd) {
        const float kt = io<IO>::load(k + t * a.k.stride + d);
        const float qt = io<IO>::load(q + t * a.q.stride + d);
        if (TAN) ds[e] = decay * (ds[e] + s[e]);
        if (!a.rev) s[e] *= decay;
        s[e] = __builtin_fmaf(vt * a.write_scale, kt, s[e]);
        dot = __builtin_fmaf(TAN ? ds[e] : s[e], qt, dot);
        if (a.rev) s[e] *= decay;
      }
    }
    for (int m = 1; m < 8; m <<= 1) dot += __shfl_xor(dot, m);
    if (TAN) {
      if (on && c == 0)
        dg = __builtin_fmaf(dot * a.read_scale,
                            io<IO>::load(static_cast<const IO*>(a.dy.p) + t * a.dy.stride +
                                         (int64_t)(head / a.dy.hdiv) * a.vd + row), dg);
    } else if (on && c == 0) {
      const int64_t at = (t * a.heads + head) * a.vd + row;
      if (a.o_f32) static_cast<float*>(a.o)[at] = dot * a.read_scale;
      else io<IO>::store(static_cast<IO*>(a.o) + at, dot * a.read_scale);
    }
  }
  if (TAN) {
    __shared__ float part[256];
    if (a.ds_last && on)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = e * 8 + c;
        if (d < a.kd) dg = __builtin_fmaf(ds[e], a.ds_last[(sh * a.vd + row) * a.kd + d], dg);
      }
    part[threadIdx.x] = dg;
    __syncthreads();
    if (threadIdx.x == 0) {
      float sum = 0.0f;
      for (int i = 0; i < 256; ++i) sum += part[i];
      a.dg_part[(seq * vblocks + blockIdx.x % vblocks) * a.heads + head] = sum;
    }
    return;
  }
  if (!a.s_last || !on) return;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int d = e * 8 + c;
    if (d < a.kd) a.s_last[(sh * a.vd + row) * a.kd + d] = s[e];
  }
}

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

template <typename IO, int E>
void launch_walk(const LinArgs& a, dim3 grid, int vblocks, hipStream_t stream) {
  if (a.dg_part)
    hipLaunchKernelGGL((linattn_walk_kernel<IO, E, true>), grid, dim3(256), 0, stream, a, vblocks);
  else
    hipLaunchKernelGGL((linattn_walk_kernel<IO, E, false>), grid, dim3(256), 0, stream, a, vblocks);
}

template <typename IO> hipError_t launch_io(const LinArgs& a, hipStream_t stream) {
  const int vblocks = (a.vd + 31) / 32;
  const dim3 grid((unsigned)(a.nseq * a.heads * vblocks));
  if (a.kd <= 64) launch_walk<IO, 8>(a, grid, vblocks, stream);
  else if (a.kd <= 128) launch_walk<IO, 16>(a, grid, vblocks, stream);
  else launch_walk<IO, 32>(a, grid, vblocks, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linattn(const LinArgs* walks, int n, bool io_bf16, hipStream_t stream) {
  if (io_bf16) return launch_linattn_mm(walks, n, stream);
  for (int i = 0; i < n; ++i) {
    const hipError_t e = launch_io<float>(walks[i], stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

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
