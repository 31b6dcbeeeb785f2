// ssm_linattn_step.hip -- one token of the linear attention with a decay per
// head, on a resident fp32 state (gfx950, wave64):
//   S <- exp(log_decay) S + v k^T,   o = scale S q,   S [vdim, kdim] in place.
//
// Bound by HBM: the state is read and written once (2 * vdim * kdim * 4 bytes
// a head and sequence) and everything else is small.  Eight lanes own a row of
// the state, each a float4 of every 32 channels, so that one load of a wave
// covers eight rows of 128 contiguous bytes; a wave takes R groups of eight
// rows with all their loads in flight.  The row's dot with q is summed over
// the eight lanes by DPP exchanges.  Measured: 256 sequences x 40 heads of 128 x
// 128 (1.34 GB of states) 239 us, 5.6 TB/s, past the 4.9 TB/s of a large copy;
// 4 sequences take as long as the call.
#include <algorithm>

#include "ssm_device.h"
#include "ssm_linattn.h"

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
__global__ __launch_bounds__(256) void linattn_step_kernel(LinStepArgs a, int waves_per_head,
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
  const float decay = fast_exp2(a.log_decay[head] * kLog2e);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool on = row0 + 8 * r < a.vd;
    const float v = on ? io<IO>::load(vp + 8 * r) : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int d = 32 * f + 4 * c;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[r][f][i] = __builtin_fmaf(decay, s[r][f][i], v * k[f][i]);
        dot = __builtin_fmaf(s[r][f][i], q[f][i], dot);
      }
      if (on && d < a.kd)
        __builtin_nontemporal_store(s[r][f], reinterpret_cast<v4f*>(h + 8 * r * a.kd + d));
    }
    dot = sum8(dot);
    if (on && c == 0) io<IO>::store(o + row0 + 8 * r, dot * a.scale);
  }
}

template <typename IO, int F>
hipError_t launch_f(const LinStepArgs& a, hipStream_t stream) {
  constexpr int R = F <= 4 ? 4 : 2;
  const int wph = (a.vd + 8 * R - 1) / (8 * R);
  const int64_t blocks = (a.batch * a.heads * wph + 3) / 4;
  for (int64_t b = 0; b < blocks; b += max_blocks(256)) {
    const dim3 grid((unsigned)std::min<int64_t>(blocks - b, max_blocks(256)));
    hipLaunchKernelGGL((linattn_step_kernel<IO, F, R>), grid, dim3(256), 0, stream, a, wph, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename IO> hipError_t launch_io(const LinStepArgs& a, hipStream_t stream) {
  switch ((a.kd + 31) / 32) {
    case 1: return launch_f<IO, 1>(a, stream);
    case 2: return launch_f<IO, 2>(a, stream);
    case 3: return launch_f<IO, 3>(a, stream);
    case 4: return launch_f<IO, 4>(a, stream);
    case 5: case 6: return launch_f<IO, 6>(a, stream);
    default: return launch_f<IO, 8>(a, stream);
  }
}

}  // namespace

hipError_t launch_linattn_step(const LinStepArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_io<bf16>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace ssm
