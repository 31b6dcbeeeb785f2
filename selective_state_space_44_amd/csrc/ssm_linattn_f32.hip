// ssm_linattn_f32.hip -- linear attention with one decay per head for fp32
// operands (gfx950, wave64), on the fp32 matrix instructions: the chunked walk
// of ssm_linattn_mm.hip in chunks of 32 tokens with every product in fp32, so
// nothing is split or rounded on the way.
//
// A block of four waves walks one unit of one head; each wave owns 16 value
// channels with the whole key dimension of their state in its accumulators.
// v_mfma_f32_16x16x4: lane l, g = l / 16: A row l % 16 and B column l % 16 of
// contraction index g; result column l % 16, rows 4 g..4 g + 3.  Contraction
// indices are taken in the order i, 4 + i, 8 + i, 12 + i of each 16, so that a
// lane's four consecutive floats serve four instructions and an accumulator
// tile is an operand as it stands.
//
// Bound by the matrix instructions (64 flops a cycle and SIMD, a sixteenth of
// the bf16 rate) and, with few blocks, by latency.  Measured: 3 x 517 tokens of
// 24 heads of 64, from given states: 30 us (8 at the copy rate), backward 48, with
// the decay's gradient 125; 300 heads over 4096 tokens of 64: 423 us, 48 TFLOP/s;
// 4 x 4096 tokens, 40 heads over 8, of 128: 650 us, backward 1700 (63 TFLOP/s),
// with the decay's gradient 3100.  In chunks of 32 a block's q, k, v and P
// at keys of 128 take 47 KB of LDS, three blocks to a CU.
#include <algorithm>

#include "ssm_linattn_walk.h"

namespace ssm {
namespace {

constexpr int C = 32;  // tokens of a chunk; a segment is whole chunks
constexpr int kWaves = 4, kThreads = 64 * kWaves, VB = 16 * kWaves;
static_assert(kLinChunk % C == 0, "segments are whole chunks");

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f4 mfma4(float a, float b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4 lds4(const float* p) { return *reinterpret_cast<const f4*>(p); }

// A [C, W] tile on its way into LDS, rows W + 4 floats apart there.
template <int W> struct Tile {
  static constexpr int kPerRow = W / 4, kRows = kThreads / kPerRow, kPasses = C / kRows;
  static constexpr int kStride = W + 4;
  f4 r[kPasses];
  __device__ __forceinline__ static uint32_t start(int64_t stride, int col0, int dim) {
    const int c = (threadIdx.x % kPerRow) * 4 + col0;
    return c < dim ? (threadIdx.x / kPerRow) * (uint32_t)stride * 4 + (uint32_t)c * 4 : 0x7f000000u;
  }
  // Rows 0..n-1 from `base`, in memory order; rows past n read zero.
  __device__ __forceinline__ void load(const float* base, int64_t stride, int n, int dim,
                                       uint32_t start) {
    const uint32_t sb = (uint32_t)stride * 4;
    const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(base, (uint32_t)(n - 1) * sb + (uint32_t)dim * 4);
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      r[p] = __builtin_bit_cast(
          f4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, start + p * kRows * sb, 0, 0));
  }
  __device__ __forceinline__ void store(float* lds) const {
    const int c = (threadIdx.x % kPerRow) * 4, row = threadIdx.x / kPerRow;
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      *reinterpret_cast<f4*>(lds + (row + p * kRows) * kStride + c) = r[p];
  }
};

template <int KD, bool MAIN, bool TAN> struct alignas(16) Shared {
  float k[C * Tile<KD>::kStride];
  float v[C * Tile<VB>::kStride];
  float q[MAIN ? C * Tile<KD>::kStride : 4];
  float p[MAIN ? C * (C + 4) : 4];  // [t][s]
  float w[C], rw[C];                // weights by row, as in ssm_linattn_mm.hip
  double part[TAN ? kThreads : 2];  // sums of the block's threads
  int odd[2];
};

template <int KD, bool MAIN, bool REV, bool TAN>
__device__ __forceinline__ void walk(const LinArgs& a, Shared<KD, MAIN, TAN>& sh, const Unit& x,
                                     uint32_t u, int head, int vb0, uint32_t part_at) {
  constexpr int RT = KD / 16, QS = Tile<KD>::kStride, VS = Tile<VB>::kStride, PS = C + 4;
  const bool last_unit = x.p0 + x.n >= x.len;
  if (!MAIN && last_unit) return;

  const int64_t uh = (int64_t)u * a.heads + head;
  const int w = wave_id(), lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  const float g2 = log2_decay(a.log_decay[head]);
  const int dv0 = w * 16, dvs = vb0 + dv0 + r16;

  // S[rt]: keys 16 rt + 4 g + i of the wave's channel r16
  f4 S[RT], T[TAN ? RT : 1];
  const int64_t state = (int64_t)a.vd * a.kd, seq_state = ((int64_t)x.seq * a.heads + head) * state;
  const uint32_t state_bytes = (uint32_t)state * 4;
  auto place = [&](int rt) {
    const int dk = 16 * rt + 4 * g;
    return dvs < a.vd && dk < a.kd ? (uint32_t)(dvs * a.kd + dk) * 4 : 0x7f000000u;
  };
  auto load_state = [&](const float* from, bool some, f4* to) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(from, some ? state_bytes : 0u);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      to[rt] = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(rs, place(rt), 0, 0));
  };
  auto store_state = [&](float* to, const f4* from) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(to, state_bytes);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      __builtin_amdgcn_raw_buffer_store_b128(
          __builtin_bit_cast(u4, from[rt]), rs, place(rt),
          0, 0);
  };
  // what enters the segment; folded, the first segment's end
  const bool inner = MAIN && x.p0 > 0;
  const int64_t entry = (uh - (a.fold ? (int64_t)x.seg * a.heads : 0)) * state;
  if (x.seg == 0 && a.s0 && a.s0_swap) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.s0 + seq_state, state_bytes);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int dk = 16 * rt + 4 * g + i;
        S[rt][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            rs, dvs < a.vd && dk < a.kd ? (uint32_t)(dk * a.vd + dvs) * 4 : 0x7f000000u, 0, 0));
      }
  } else {
    load_state(inner ? a.ws_state + entry : a.s0 + seq_state, inner || (x.seg == 0 && a.s0), S);
  }
  if constexpr (TAN) load_state(a.ws_tangent + entry, inner, T);
  if (MAIN && x.seg > 1 && a.fold) {  // join the segments between
    const Decays all = wave_decays(a.log_decay[head], x.seg_len);
    for (int j = x.seg - 1; j > 0; --j) {
      const float as = decay_of(all, x.seg - 1 - j);
      const int64_t slot = (uh - (int64_t)j * a.heads) * state;
      f4 own[RT];
      if constexpr (TAN) {
        load_state(a.ws_tangent + slot, true, own);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          T[rt] = as * (T[rt] + (float)x.seg_len * S[rt]) + own[rt];
      }
      load_state(a.ws_state + slot, true, own);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[rt][i] = __builtin_fmaf(as, S[rt][i], own[rt][i]);
    }
  }

  const float* qp = static_cast<const float*>(a.q.p) + (int64_t)(head / a.q.hdiv) * a.kd;
  const float* kp = static_cast<const float*>(a.k.p) + (int64_t)(head / a.k.hdiv) * a.kd;
  const float* vp = static_cast<const float*>(a.v.p) + (int64_t)(head / a.v.hdiv) * a.vd;
  const uint32_t q_at = Tile<KD>::start(a.q.stride, 0, a.kd);
  const uint32_t k_at = Tile<KD>::start(a.k.stride, 0, a.kd);
  const uint32_t v_at = Tile<VB>::start(a.v.stride, vb0, a.vd);
  auto token0 = [&](int c0, int n) { return x.first + (REV ? x.len - c0 - n : c0); };
  Tile<KD> tq, tk;
  Tile<VB> tv;
  auto load = [&](int c0, int n) {
    const uint32_t t0 = (uint32_t)token0(c0, n);
    if constexpr (MAIN) tq.load(qp + (uint64_t)t0 * (uint32_t)a.q.stride, a.q.stride, n, a.kd, q_at);
    tk.load(kp + (uint64_t)t0 * (uint32_t)a.k.stride, a.k.stride, n, a.kd, k_at);
    tv.load(vp + (uint64_t)t0 * (uint32_t)a.v.stride, a.v.stride, n, a.vd, v_at);
  };
  const int end = x.p0 + x.n;
  auto size = [&](int c0) { return end - c0 < C ? end - c0 : C; };
  // of whole chunks, where there are several
  const float g_chunk = scalar(power(g2, C));
  Decays chunk_decays{g_chunk, g_chunk, 0.0f};
  if (x.n > C) chunk_decays = wave_decays(a.log_decay[head], C);
  double dg = 0.0;  // the lane's part of the sum (TAN): in 64 bits over the chunks
  if (MAIN && threadIdx.x < 2) sh.odd[threadIdx.x] = 0;
  if (x.n > 0) load(x.p0, size(x.p0));
  lds_barrier();  // odd is cleared
  for (int c0 = x.p0; c0 < end; c0 += C) {
    const int n = size(c0), parity = ((c0 - x.p0) / C) & 1;
    if (c0 > x.p0) lds_barrier();  // the previous chunk's tiles are read
    if constexpr (MAIN) tq.store(sh.q);
    tk.store(sh.k);
    tv.store(sh.v);
    if constexpr (MAIN) {
      uint32_t most = 0;  // infinities and NaN: the largest exponent
#pragma unroll
      for (int p = 0; p < Tile<VB>::kPasses; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          most = max(most, __float_as_uint(tv.r[p][i]) & 0x7fffffffu);
      if (most >= 0x7f800000u) sh.odd[parity] = 1;
    }
    if (threadIdx.x < C) {
      const int i = threadIdx.x, left = i < n ? n - 1 - i : 0;
      // rows past n are no tokens; a growing decay's power may be infinite there
      sh.w[i] = i < n ? power(g2, REV ? i + 1 : left) * a.write_scale : 0.0f;
      sh.rw[i] = i < n ? power(g2, REV ? left : i + 1) * a.read_scale : 0.0f;
    }
    lds_barrier();
    if (c0 + C < end) load(c0 + C, size(c0 + C));

    const float an = n == C ? decay_of(chunk_decays, (c0 - x.p0) / C) : power(g2, n);
    if constexpr (MAIN) {
      // P: tiles (0, 0), (1, 0), (1, 1) (going back (0, 1)) of waves 0..2, the
      // fourth tile, which has no pair in walk order, zero
      if (w < 3) {
        const int tt = w == 0 ? 0 : w == 1 ? !REV : 1, st = w == 0 ? 0 : w == 1 ? REV : 1;
        f4 m{0, 0, 0, 0};
        const float* kr = sh.k + (16 * st + r16) * QS + 4 * g;
        const float* qr = sh.q + (16 * tt + r16) * QS + 4 * g;
#pragma unroll
        for (int c = 0; c < RT; ++c) {
          const f4 kv = lds4(kr + 16 * c), qv = lds4(qr + 16 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) m = mfma4(kv[i], qv[i], m);
        }
        const int ts = 16 * (tt - st) + r16 - 4 * g;
        f4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int d = REV ? j - ts : ts - j;
          const float pw = power(g2, d > 0 ? d : 0) * (TAN ? a.pair_scale * (float)d : a.pair_scale);
          // going back, rows past n come before t
          v[j] = d >= 0 && (!REV || 16 * st + 4 * g + j < n) ? m[j] * pw : 0.0f;
        }
        *reinterpret_cast<f4*>(sh.p + (16 * tt + r16) * PS + 16 * st + 4 * g) = v;
      } else {
        const int tt = REV ? 1 : 0, st = REV ? 0 : 1;
        *reinterpret_cast<f4*>(sh.p + (16 * tt + r16) * PS + 16 * st + 4 * g) = f4{0, 0, 0, 0};
      }
    }
    f4 acc[2], tan[TAN ? 2 : 1];
    if constexpr (MAIN) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        acc[tt] = f4{0, 0, 0, 0};
        if constexpr (TAN) tan[tt] = f4{0, 0, 0, 0};
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          const f4 qv = lds4(sh.q + (16 * tt + r16) * QS + 16 * rt + 4 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[tt] = mfma4(S[rt][i], qv[i], acc[tt]);
            if constexpr (TAN) tan[tt] = mfma4(T[rt][i], qv[i], tan[tt]);
          }
        }
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        if constexpr (TAN) acc[tt] = (float)(16 * tt + r16 + 1) * acc[tt] + tan[tt];
        acc[tt] *= sh.rw[16 * tt + r16];
      }
      lds_barrier();  // P is whole
      if (threadIdx.x == 0) sh.odd[parity ^ 1] = 0;
    }
    // v of the wave's channel r16, tokens 16 c + 4 g + i
    f4 vo[2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) vo[c][i] = sh.v[(16 * c + 4 * g + i) * VS + dv0 + r16];
    int first = REV ? -1 : C;  // of channel r16, the first token (in walk order) with an odd value
    bool odd = false;
    if constexpr (MAIN) {
      // as in ssm_linattn_mm.hip: an infinity or NaN must not reach an earlier
      // token through its zero weight
      odd = __builtin_amdgcn_readfirstlane(sh.odd[parity]) != 0;
      f4 vz[2] = {vo[0], vo[1]};
      if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((__float_as_uint(vo[c][i]) & 0x7f800000u) == 0x7f800000u) {
              const int s = 16 * c + 4 * g + i;
              first = REV ? max(first, s) : min(first, s);
              vz[c][i] = 0.0f;
            }
#pragma unroll
        for (int m = 16; m < 64; m <<= 1) {
          const int other = __shfl_xor(first, m);
          first = REV ? max(first, other) : min(first, other);
        }
      }
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const f4 pv = lds4(sh.p + (16 * tt + r16) * PS + 16 * c + 4 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[tt] = mfma4(vz[c][i], pv[i], acc[tt]);
        }
      if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int f = __shfl(first, 4 * g + i);
#pragma unroll
          for (int tt = 0; tt < 2; ++tt)
            if (REV ? 16 * tt + r16 <= f : 16 * tt + r16 >= f)
              acc[tt][i] = __uint_as_float(0x7fc00000u);
        }
      }
      const int dv = vb0 + dv0 + 4 * g;
      if constexpr (TAN) {
        const uint32_t row = (uint32_t)a.dy.stride * 4;
        const __amdgpu_buffer_rsrc_t ry = make_rsrc(
            static_cast<const float*>(a.dy.p) +
                (uint64_t)(uint32_t)token0(c0, n) * (uint32_t)a.dy.stride + (int64_t)head * a.vd,
            (uint32_t)(n - 1) * row + (uint32_t)a.vd * 4);
        const uint32_t ya = dv < a.vd ? r16 * row + (uint32_t)dv * 4 : 0x7f000000u;
        float here = 0.0f;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          const f4 y = __builtin_bit_cast(
              f4, __builtin_amdgcn_raw_buffer_load_b128(ry, ya + 16 * tt * row, 0, 0));
          if (16 * tt + r16 < n && dv < a.vd)
#pragma unroll
            for (int i = 0; i < 4; ++i) here = __builtin_fmaf(acc[tt][i], y[i], here);
        }
        dg += (double)here;
      } else {
        const uint32_t row = (uint32_t)a.heads * a.vd * 4;
        const __amdgpu_buffer_rsrc_t ro =
            make_rsrc(static_cast<float*>(a.o) + ((int64_t)token0(c0, n) * a.heads + head) * a.vd,
                      (uint32_t)(n - 1) * row + (uint32_t)a.vd * 4);
        const uint32_t oa = dv < a.vd ? r16 * row + (uint32_t)dv * 4 : 0x7f000000u;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
          __builtin_amdgcn_raw_buffer_store_b128(
              __builtin_bit_cast(u4, acc[tt]), ro,
              oa + 16 * tt * row, 0, 0);
      }
    }

    // S <- a^n S + k^T (w v).  The chunk's terms are added up first: four tokens
    // at a time their part of T would be below its rounding after many chunks
    // (65536 tokens at decays near 1: 1.5e-4 of the decay's gradient).
    f4 wv[2], tv_[TAN ? 2 : 1];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      wv[c] = vo[c] * lds4(sh.w + 16 * c + 4 * g);
      if constexpr (TAN) {
#pragma unroll
        for (int i = 0; i < 4; ++i) tv_[c][i] = wv[c][i] * (float)(n - 1 - (16 * c + 4 * g + i));
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      f4 d{0, 0, 0, 0}, td{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float kv = sh.k[(16 * c + 4 * g + i) * QS + 16 * rt + r16];
          d = mfma4(kv, wv[c][i], d);
          if constexpr (TAN) td = mfma4(kv, tv_[c][i], td);
        }
      if constexpr (TAN) T[rt] = an * (T[rt] + (float)n * S[rt]) + td;
#pragma unroll
      for (int i = 0; i < 4; ++i) S[rt][i] = __builtin_fmaf(an, S[rt][i], d[i]);
    }
    if (MAIN && __builtin_expect(odd, 0) && (REV ? first >= 0 : first < C)) {
      const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        S[rt] = f4{nan, nan, nan, nan};
        if constexpr (TAN) T[rt] = S[rt];
      }
    }
  }

  if constexpr (MAIN && TAN) {
    if (a.ds_last && last_unit) {
      f4 d[RT];
      load_state(a.ds_last + seq_state, true, d);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) dg += (double)(T[rt][i] * d[rt][i]);
    }
    sh.part[threadIdx.x] = dg;
    __syncthreads();
    for (int m = kThreads / 2; m > 0; m >>= 1) {
      if ((int)threadIdx.x < m) sh.part[threadIdx.x] += sh.part[threadIdx.x + m];
      __syncthreads();
    }
    if (threadIdx.x == 0) a.dg_part[part_at] = (float)sh.part[0];
  }
  // the result, or a segment's end for those after it
  const bool between = !last_unit && (!MAIN || (a.lead && x.seg == 0));
  if (!between && (TAN || !last_unit || !a.s_last)) return;
  store_state(between ? a.ws_state + uh * state : a.s_last + seq_state, S);
  if constexpr (TAN) store_state(a.ws_tangent + uh * state, T);
}

// LDS of a pass' blocks: of walks, of states, of either.
template <int KD, Pass PASS, bool TAN> union Storage {
  Shared<KD, PASS != kState, TAN> main;
  Shared<KD, false, TAN> state;
};

// The r-th block of a walk, as in ssm_linattn_mm.hip.
template <int KD, Pass PASS, bool TAN>
__device__ __forceinline__ void walk_block(const LinArgs& a, Storage<KD, PASS, TAN>& sh, uint32_t vblocks,
                                           uint32_t r, Places at) {
  if (r >= at.count * (uint32_t)a.heads * vblocks) return;
  const uint32_t ph = r / vblocks, vb = r - ph * vblocks, place = ph / (uint32_t)a.heads;
  const uint32_t u = unit_at(a, at.first + place);
  const int head = (int)(ph - place * (uint32_t)a.heads), vb0 = (int)vb * VB;
  const uint32_t part_at = (u * vblocks + vb) * (uint32_t)a.heads + (uint32_t)head;
  Unit x;
  if (!unit_of(a, u, x)) {
    if (TAN && PASS == kWalk && threadIdx.x == 0) a.dg_part[part_at] = 0.0f;
    return;
  }
  if (PASS == kWalk && a.lead && x.seg == 0) return;
  if constexpr (PASS != kWalk) {
    if (PASS == kState || x.seg > 0) {
      if (!TAN && a.rev)
        walk<KD, false, !TAN, TAN>(a, sh.state, x, u, head, vb0, part_at);
      else
        walk<KD, false, false, TAN>(a, sh.state, x, u, head, vb0, part_at);
      return;
    }
  }
  if constexpr (PASS != kState) {
    if (!TAN && a.rev)
      walk<KD, true, !TAN, TAN>(a, sh.main, x, u, head, vb0, part_at);
    else
      walk<KD, true, false, TAN>(a, sh.main, x, u, head, vb0, part_at);
  }
}

template <int KD, Pass PASS>
__global__ __launch_bounds__(kThreads, 2) void linattn_f32_kernel(LinWalks ws, uint32_t vblocks,
                                                                  Places at, uint32_t group) {
  __shared__ Storage<KD, PASS, false> sh;
  const uint32_t block = xcd_block(blockIdx.x, group), r = block / (uint32_t)ws.n;
  walk_block<KD, PASS, false>(ws.a[block - r * (uint32_t)ws.n], sh, vblocks, r, at);
}

template <int KD, Pass PASS>
__global__ __launch_bounds__(kThreads, KD > 128 ? 1 : 2) void linattn_f32_tan_kernel(
    LinArgs a, uint32_t vblocks, Places at, uint32_t group) {
  __shared__ Storage<KD, PASS, true> sh;
  walk_block<KD, PASS, true>(a, sh, vblocks, xcd_block(blockIdx.x, group), at);
}

template <int KD, Pass PASS> hipError_t launch_pass(const LinWalks& ws, hipStream_t stream) {
  const LinArgs& a = ws.a[0];
  const uint32_t vblocks = (uint32_t)((a.vd + VB - 1) / VB);
  const Places all = places_of(a, PASS);
  const uint32_t per = (uint32_t)a.heads * vblocks * (uint32_t)ws.n;  // blocks of a place
  const uint32_t shared = (uint32_t)std::max({a.q.hdiv, a.k.hdiv, a.v.hdiv});
  const uint32_t group = std::min(shared * vblocks * (uint32_t)ws.n, kMaxGroup);
  for (uint32_t done = 0; done < all.count;) {
    const Places at = slice_of(all, done, kThreads, per, 8 * kMaxGroup);
    const dim3 grid((at.count * per + 8 * group - 1) / (8 * group) * (8 * group)), threads(kThreads);
    if (a.dg_part) {
      if constexpr (PASS != kLead)
        hipLaunchKernelGGL((linattn_f32_tan_kernel<KD, PASS>), grid, threads, 0, stream, a, vblocks,
                           at, group);
    } else {
      hipLaunchKernelGGL((linattn_f32_kernel<KD, PASS>), grid, threads, 0, stream, ws, vblocks, at,
                         group);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    done += at.count;
  }
  return hipSuccess;
}

template <int KD> hipError_t launch_kd(const LinWalks& ws, hipStream_t stream) {
  if (ws.a[0].seg_len) {
    hipError_t e = ws.a[0].lead ? launch_pass<KD, kLead>(ws, stream)
                                : launch_pass<KD, kState>(ws, stream);
    if (e == hipSuccess && !ws.a[0].fold) e = launch_lin_carry(ws, stream);
    if (e != hipSuccess) return e;
  }
  return launch_pass<KD, kWalk>(ws, stream);
}

}  // namespace

hipError_t launch_linattn_f32(const LinArgs* walks, int n, hipStream_t stream) {
  LinWalks ws{};
  ws.n = n;
  for (int i = 0; i < n; ++i) ws.a[i] = walks[i];
  const int kd = walks[0].kd;
  if (kd <= 64) return launch_kd<64>(ws, stream);
  if (kd <= 128) return launch_kd<128>(ws, stream);
  return launch_kd<256>(ws, stream);
}

}  // namespace ssm
