// ssm_delta_spans.hip -- the states between the spans of a sequence in the gated delta
// rule (gfx950, wave64): E_j = L_j + E_(j-1) W_j for the spans j from the second to the
// last but one, in place of the L_j (ssm_delta_walk.h); of a backward's adjoints
// F_(j-1) = L'_(j-1) + F_j W_j^T, from the last but one to the second.  W = X + dec 1,
// with dec in two fp32 parts: as one matrix of fp32 numbers, hundreds of spans of like
// decays would round it alike (1.5e-5 over 256).  So would they the states: what a state
// loses as it is rounded goes with it to the next one.
//
// A block takes 16 rows of a head's states through all spans; each of its four waves
// has every fourth tile of 16 columns.  fp32 matrix instructions: E keeps its 24 bits.
#include <algorithm>

#include "ssm_delta_mm.h"

namespace ssm {
namespace {

template <int KD, bool BACK> __device__ __forceinline__ void span_states(const DeltaArgs& a, float* sh) {
  constexpr int TILES = KD / 64, LD = KD + 4;  // a wave's tiles; rows in LDS, no bank twice
  const int w = wave_id(), lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  const int seq = (int)(blockIdx.y / (uint32_t)a.heads), head = (int)(blockIdx.y - (uint32_t)(seq * a.heads));
  const SpanAt at0 = spans_of_seq(a, seq);
  const int inner = at0.n - 2;  // spans with a W: from the second on
  if (inner < 1) return;
  const int64_t unit = (int64_t)(at0.first - seq) * a.heads + head, state = (int64_t)a.vd * a.kd,
                move = delta_move_floats(a.kd);
  const int row0 = blockIdx.x * 16;
  auto state_of = [&](int j) { return (BACK ? a.span_backs : a.span_ends) + (unit + (int64_t)j * a.heads) * state; };
  const uint32_t state_bytes = (uint32_t)state * 4, move_bytes = (uint32_t)(a.kd * a.kd) * 4;
  auto at = [&](int row, int rows, int col) {
    return row < rows && col < a.kd ? (uint32_t)(row * a.kd + col) * 4 : 0x7f000000u;
  };
  auto load = [](__amdgpu_buffer_rsrc_t rs, uint32_t from) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, from, 0, 0));
  };
  {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(state_of(BACK ? inner : 0), state_bytes);
    for (int i = threadIdx.x; i < 16 * KD; i += 256)
      sh[i / KD * LD + i % KD] = load(rs, at(row0 + i / KD, a.vd, i % KD));
  }
  __syncthreads();
  float low[TILES][4] = {};  // what E has less than the states, of the lane's places in acc
  for (int i = 0; i < inner; ++i) {
    const int j = BACK ? inner - i : i + 1;  // the span
    const float* w_at = a.span_moves + (unit + (int64_t)j * a.heads) * move;
    const float dec = w_at[a.kd * a.kd], dec_low = w_at[a.kd * a.kd + 1];
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(w_at, move_bytes),
                                 re = make_rsrc(state_of(BACK ? j - 1 : j), state_bytes);
    float b[TILES][KD / 4];
    f32x4_t acc[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int col = 16 * (w + 4 * t) + r16;
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[t][x] = load(re, at(row0 + 4 * g + x, a.vd, col));
#pragma unroll
      for (int k = 0; k < KD / 4; ++k)
        b[t][k] = load(rw, BACK ? at(col, a.kd, 4 * k + g) : at(4 * k + g, a.kd, col));
    }
#pragma unroll
    for (int k = 0; k < KD / 4; ++k) {
      const float e = sh[r16 * LD + 4 * k + g];
#pragma unroll
      for (int t = 0; t < TILES; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(e, b[t][k], acc[t], 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int col = 16 * (w + 4 * t) + r16;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
#pragma clang fp contract(off)  // (the remainders of a product and of a sum, exact)
        const float e = sh[(4 * g + x) * LD + col], most = dec * e;
        const float rest = acc[t][x] + __builtin_fmaf(dec_low, e, __builtin_fmaf(dec, low[t][x], __builtin_fmaf(dec, e, -most)));
        const float sum = most + rest, taken = sum - most, lost = (most - (sum - taken)) + (rest - taken);
        acc[t][x] = sum;
        low[t][x] = __builtin_isfinite(lost) ? lost : 0.0f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int col = 16 * (w + 4 * t) + r16;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        sh[(4 * g + x) * LD + col] = acc[t][x];
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[t][x]), re,
                                              at(row0 + 4 * g + x, a.vd, col), 0, 0);
      }
    }
    __syncthreads();
  }
}

template <int KD> __global__ __launch_bounds__(256) void delta_span_states_kernel(DeltaArgs a) {
  __shared__ float sh[16 * (KD + 4)];
  if (blockIdx.z) span_states<KD, true>(a, sh);
  else span_states<KD, false>(a, sh);
}

}  // namespace

hipError_t launch_delta_span_states(const DeltaArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.vd + 15) / 16), (unsigned)(a.nseq * a.heads), a.back ? 2 : 1);
  if (a.kd <= 64) hipLaunchKernelGGL((delta_span_states_kernel<64>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((delta_span_states_kernel<128>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace ssm
