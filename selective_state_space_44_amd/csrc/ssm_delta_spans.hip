// ssm_delta_spans.hip -- the states between the spans of a sequence in the gated delta
// rule (gfx950, wave64): E_j = L_j + E_(j-1) W_j for the spans j from the second to the
// last but one, in place of the L_j (ssm_delta_walk.h); of a backward's adjoints
// F_(j-1) = L'_(j-1) + F_j W_j^T, from the last but one to the second.  W = X + dec 1,
// with dec in two fp32 parts: as one matrix of fp32 numbers, hundreds of spans of like
// decays would round it alike (1.5e-5 over 256).  So would they the states, which go on
// in 64 bits.
//
// A block takes 16 rows of a head's states through all spans; each of its four waves
// has a quarter of the columns.  fp32 matrix instructions: E keeps its 24 bits.
#include <algorithm>

#include "ssm_delta_mm.h"

namespace ssm {
namespace {

template <int KD, bool BACK> __device__ __forceinline__ void span_states(const DeltaArgs& a, float* sh) {
  constexpr int TILES = KD / 64, LD = KD + 4;  // a wave's tiles; rows in LDS
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
  // A lane's columns of the result, one of each of the wave's tiles (kdim is a multiple of
  // 8), and of the 16 m + 4 g + 0..3 that it sums over four at a time.
  struct alignas(4 * TILES) Cols {
    float v[TILES];
  };
  const int col = TILES * (16 * w + r16);
  auto load = [](__amdgpu_buffer_rsrc_t rs, uint32_t from) {
    if constexpr (TILES == 1) return __builtin_bit_cast(Cols, __builtin_amdgcn_raw_buffer_load_b32(rs, from, 0, 0));
    else return __builtin_bit_cast(Cols, __builtin_amdgcn_raw_buffer_load_b64(rs, from, 0, 0));
  };
  // What a step reads besides the state: W by the lane's operands, and L.  All of it is
  // asked for one step ahead, and stays as it comes (moved, it would be waited for).
  struct Operands {
    float b[TILES][KD / 4], dec, dec_low;
    Cols l[4];
  };
  auto span_of = [&](int i) { return BACK ? inner - i : i + 1; };
  auto resource = [&](int i) {  // (beyond the last: over no memory)
    return make_rsrc(state_of(span_of(i) - (BACK ? 1 : 0)), i < inner ? state_bytes : 0);
  };
  auto move_of = [&](int i) { return a.span_moves + (unit + (int64_t)span_of(i) * a.heads) * move; };
  const uint32_t w_at = at(0, 1, col) + (uint32_t)(4 * g * a.kd) * 4;  // (rows past the last: beyond W)
  auto ask = [&](int i, Operands& o) {
    const __amdgpu_buffer_rsrc_t re = resource(i),
                                 rw = make_rsrc(move_of(i), i < inner ? move_bytes : 0),
                                 rd = make_rsrc(move_of(i) + a.kd * a.kd, i < inner ? 8 : 0);
#pragma unroll
    for (int m = 0; m < KD / 16; ++m) {
      if constexpr (BACK) {
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          const f32x4_t r = __builtin_bit_cast(
              f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, at(col + t, a.kd, 16 * m + 4 * g), 0, 0));
#pragma unroll
          for (int x = 0; x < 4; ++x) o.b[t][4 * m + x] = r[x];
        }
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const Cols r = load(rw, w_at + (uint32_t)((16 * m + x) * a.kd) * 4);
#pragma unroll
          for (int t = 0; t < TILES; ++t) o.b[t][4 * m + x] = r.v[t];
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) o.l[x] = load(re, at(row0 + 4 * g + x, a.vd, col));
    o.dec = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rd, 0, 0, 0));
    o.dec_low = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rd, 4, 0, 0));
    __builtin_amdgcn_sched_barrier(0);  // (before the step's products, not after)
  };
  double E[TILES][4];  // the lane's places of the state
  auto step = [&](int i, Operands& o) {
    const float* from = sh + (i & 1) * 16 * LD;
    float* to = sh + (~i & 1) * 16 * LD;
    f32x4_t acc[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < KD / 16; ++m) {
      const f32x4_t e = *reinterpret_cast<const f32x4_t*>(from + r16 * LD + 16 * m + 4 * g);
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int t = 0; t < TILES; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(e[x], o.b[t][4 * m + x], acc[t], 0, 0, 0);
    }
    const __amdgpu_buffer_rsrc_t re = resource(i);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      Cols now;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        E[t][x] = __builtin_fma((double)o.dec + (double)o.dec_low, E[t][x], (double)(acc[t][x] + o.l[x].v[t]));
        now.v[t] = (float)E[t][x];
      }
      *reinterpret_cast<Cols*>(to + (4 * g + x) * LD + col) = now;
      const uint32_t out = at(row0 + 4 * g + x, a.vd, col);
      if constexpr (TILES == 1) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(now.v[0]), re, out, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, now), re, out, 0, 0);
    }
    lds_barrier();  // (the states in `from` are read too: the step after the next one's)
  };
  Operands even, odd;
  {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(state_of(BACK ? inner : 0), state_bytes);
    Cols first[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) first[x] = load(rs, at(row0 + 4 * g + x, a.vd, col));
    ask(0, even);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      *reinterpret_cast<Cols*>(sh + (4 * g + x) * LD + col) = first[x];
#pragma unroll
      for (int t = 0; t < TILES; ++t) E[t][x] = first[x].v[t];
    }
    lds_barrier();
  }
  for (int i = 0; i < inner; i += 2) {
    ask(i + 1, odd);
    step(i, even);
    if (i + 1 == inner) break;
    ask(i + 2, even);
    step(i + 1, odd);
  }
}

template <int KD> __global__ __launch_bounds__(256) void delta_span_states_kernel(DeltaArgs a) {
  __shared__ alignas(16) float sh[2 * 16 * (KD + 4)];
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
