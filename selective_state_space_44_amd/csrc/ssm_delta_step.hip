// ssm_delta_step.hip -- one token of the gated delta rule on a resident fp32
// state (gfx950, wave64), S [vdim, kdim] in place:
//   S <- a S,   u = beta (v - S k),   S <- S + u k^T,   o = scale S q.
//
// Bound by HBM: the state is read and written once (2 * vdim * kdim * 4 bytes a
// head and sequence) and everything else is small.  Both dots and the update are
// done while the state's rows are in registers: eight lanes own a row, each a
// float4 of every 32 channels, so that one load of a wave covers eight rows of
// 128 contiguous bytes; a wave takes R groups of eight rows with all their loads
// in flight, and sums over the eight lanes by DPP exchanges.
#include <algorithm>

#include "ssm_device.h"
#include "ssm_delta.h"

namespace ssm {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4f load4(const float* p) { return *reinterpret_cast<const v4f*>(p); }
__device__ __forceinline__ v4f load4(const bf16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return v4f{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
             __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
}

template <int CTRL> __device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// Sum over 8 consecutive lanes: quad swaps, then the row's half mirror.
__device__ __forceinline__ float sum8(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  return v + dpp<0x141>(v);
}

// F float4s of a row per lane (kd <= 32 F), R row groups per wave.
template <typename IO, int F, int R>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepArgs a, int waves_per_head,
                                                           int64_t block0) {
  const int64_t wave = (block0 + blockIdx.x) * 4 + wave_id();
  const int64_t bh = wave / waves_per_head;
  if (bh >= a.batch * a.heads) return;
  const int64_t b = bh / a.heads;
  const int head = (int)(bh - b * a.heads);
  const int lane = threadIdx.x & 63, c = lane & 7;
  const int row0 = (int)(wave - bh * waves_per_head) * 8 * R + (lane >> 3);
  const int64_t slot = a.slots ? a.slots[b] : b;
  IO* o = static_cast<IO*>(a.o) + bh * a.vd;
  if (slot < 0 || slot >= a.nslots) {  // no state: the row answers zero
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (c == 0 && row0 + 8 * r < a.vd) io<IO>::store(o + row0 + 8 * r, 0.0f);
    return;
  }
  float* h = a.h + ((slot * a.heads + head) * a.vd + row0) * a.kd;
  const IO* kp =
      static_cast<const IO*>(a.k.p) + b * a.k.stride + (int64_t)(head / a.k.hdiv) * a.kd;
  const IO* qp =
      static_cast<const IO*>(a.q.p) + b * a.q.stride + (int64_t)(head / a.q.hdiv) * a.kd;
  const IO* vp =
      static_cast<const IO*>(a.v.p) + b * a.v.stride + (int64_t)(head / a.v.hdiv) * a.vd + row0;
  v4f s[R][F];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int d = 32 * f + 4 * c;
      s[r][f] = v4f{0, 0, 0, 0};
      if (row0 + 8 * r < a.vd && d < a.kd)
        s[r][f] = __builtin_nontemporal_load(reinterpret_cast<v4f*>(h + 8 * r * a.kd + d));
    }
  v4f k[F], q[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int d = 32 * f + 4 * c;
    k[f] = q[f] = v4f{0, 0, 0, 0};
    if (d < a.kd) k[f] = load4(kp + d), q[f] = load4(qp + d);
  }
  // Channels that there are not (in the last float4 only) stay out of an infinite update
  // and decay: 0 times those is NaN.
  const bool in = 32 * (F - 1) + 4 * c < a.kd;
  const float decay = fast_exp2(a.log_decay[bh] * kLog2e), decay_in = in ? decay : 0.0f;
  const float beta = io<IO>::load(static_cast<const IO*>(a.beta) + bh);
  // (before the first store: the compiler cannot move them over it)
  float v[R];
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = row0 + 8 * r < a.vd ? io<IO>::load(vp + 8 * r) : 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool on = row0 + 8 * r < a.vd;
    float had = 0.0f;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[r][f][i] *= f + 1 < F ? decay : decay_in;
        had = __builtin_fmaf(s[r][f][i], k[f][i], had);
      }
    const float u = beta * (v[r] - sum8(had)), u_in = in ? u : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int d = 32 * f + 4 * c;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[r][f][i] = __builtin_fmaf(f + 1 < F ? u : u_in, k[f][i], s[r][f][i]);
        dot = __builtin_fmaf(s[r][f][i], q[f][i], dot);
      }
      if (on && d < a.kd)
        __builtin_nontemporal_store(s[r][f], reinterpret_cast<v4f*>(h + 8 * r * a.kd + d));
    }
    dot = sum8(dot);
    if (on && c == 0) io<IO>::store(o + row0 + 8 * r, dot * a.scale);
  }
}

template <typename IO, int F, int R>
hipError_t launch_r(const DeltaStepArgs& a, hipStream_t stream) {
  const int wph = (a.vd + 8 * R - 1) / (8 * R);
  const int64_t blocks = (a.batch * a.heads * wph + 3) / 4;
  for (int64_t b = 0; b < blocks; b += max_blocks(256)) {
    const dim3 grid((unsigned)std::min<int64_t>(blocks - b, max_blocks(256)));
    hipLaunchKernelGGL((delta_step_kernel<IO, F, R>), grid, dim3(256), 0, stream, a, wph, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Four row groups a wave, whose loads hide one another; a single one where the
// fours would leave every second CU without a block, and what counts is how soon
// the last wave is through: 1 sequence of 40 heads of 128 x 128 takes 4.1 us with
// one group and 5.3 with four, 4 of 16 heads of 128 x 256 in fp32 4.7 and 5.1, but
// 4 of 40 heads (160 blocks of fours) 6.2 and 6.1, 16 of them 15.0 and 12.4.
template <typename IO, int F>
hipError_t launch_f(const DeltaStepArgs& a, hipStream_t stream) {
  const int64_t fours = a.batch * a.heads * ((a.vd + 31) / 32);
  return fours <= 128 * 4 ? launch_r<IO, F, 1>(a, stream) : launch_r<IO, F, 4>(a, stream);
}

template <typename IO> hipError_t launch_io(const DeltaStepArgs& a, hipStream_t stream) {
  switch ((a.kd + 31) / 32) {
    case 1: return launch_f<IO, 1>(a, stream);
    case 2: return launch_f<IO, 2>(a, stream);
    case 3: return launch_f<IO, 3>(a, stream);
    default: return launch_f<IO, 4>(a, stream);  // kd <= 128
  }
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_io<bf16>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace ssm
