// ssm_delta_walk.h -- the chunked walks of the gated delta rule (gfx950, wave64):
// included by ssm_delta_mm.hip (bf16) and ssm_delta_f32.hip.
//
// With the records of ssm_delta_prep.hip, a chunk of 64 tokens that the state S
// [vd, kd] enters is five products instead of 64 rank-one updates:
//   x = v - exp(G) (k S^T),   r = (1 + N b)^-1 x,   u = b r
//   o = scale (exp(G) (q S^T) + P u),    P_ts = exp(G_t - G_s) q_t . k_s, s <= t
//   S <- exp(G_end) S + sum over s of exp(G_end - G_s) u_s k_s^T.
// The backward walks twice: forward, without o, keeping the states S and r; and
// back with the adjoint D of the state,
//   du = exp(G_end - G) (k D^T) + scale P^T dy,   y = (1 + b N)^-T du,
//   dv = b y,   D <- exp(G_end) D + scale sum of exp(G) dy q^T - sum of exp(G) dv k^T,
// keeping D and y.  From those ssm_delta_grads.hip forms the other gradients, all
// chunks at once.
//
// A block of NW waves walks one sequence of one head over 16 NW value channels.
// Each wave owns 16 of them with their whole state in registers and everything
// computed from it: a result tile is, split into bf16 parts, the operand of the
// next product (ssm_delta_mm.h), so nothing of x, r, u or S is exchanged.  In LDS
// are the chunk's tiles of k, q and v, the inverse and P, which the waves form
// together.  S and D, and what enters them, are sums of three parts (24 bits).
// o is rounded to bf16 and P and u enter it as two.
#pragma once

#include <algorithm>

#include "ssm_delta_mm.h"

namespace ssm {
namespace {

enum Walk { kForward, kKeep, kBack };  // outputs; states and r for a backward; its adjoint

__device__ __forceinline__ uint32_t xcd_block(uint32_t b, uint32_t group) {
  // Logical block number in a grid handed out round robin to the 8 XCDs: runs of
  // `group` blocks, which read the same keys, go to one XCD and share its L2.
  const uint32_t round = b / (8 * group), i = b - round * 8 * group;
  return round * 8 * group + (i & 7) * group + (i >> 3);
}

template <typename IO, int KD, int NW, Walk W> struct alignas(256) Shared {
  typedef Mat<IO> M;
  static constexpr int VB = 16 * NW, kPP = W == kBack ? M::kParts : 2;
  uint8_t k[Tile<IO, KD>::kBytes];
  uint8_t q[W == kKeep ? 16 : Tile<IO, KD>::kBytes];
  uint8_t v[Tile<IO, VB>::kBytes];  // v or dy
  uint8_t t[kDeltaFrags][M::template kFragBytes<M::kParts>];
  uint8_t p[W == kKeep ? 1 : kDeltaFrags][M::template kFragBytes<kPP>];
  float rows[kDeltaRows][C];
  float ends[4];
  int odd[2];  // whether v holds an infinity or NaN, by chunk parity
};

// 8 values by token 32 p + 8 g ..
__device__ __forceinline__ void rows8(const float* row, int p, int g, float* x) {
  const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(row + 32 * p + 8 * g);
  const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(row + 32 * p + 8 * g + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = lo[i], x[4 + i] = hi[i];
}

// A fragment of the record in the registers of a wave's lanes.
struct Frag {
  f32x4_t lo, hi;
};

template <typename IO, int KD, int NW, Walk W>
__device__ __forceinline__ void walk(const DeltaArgs& a, Shared<IO, KD, NW, W>& sh, int seq, int head,
                                     int vb0) {
  typedef Mat<IO> M;
  constexpr int VB = 16 * NW, THREADS = 64 * NW, KT = KD / 16, KS = KD / 32, NP = M::kParts;
  typedef Tile<IO, KD> KTile;
  typedef Tile<IO, VB> VTile;
  constexpr int kPP = Shared<IO, KD, NW, W>::kPP;
  constexpr bool BACK = W == kBack;
  const Seq s = seq_of(a, seq);
  const int w = wave_id(), lane = threadIdx.x & 63;
  int r16 = lane & 15, g = lane >> 4, tid = threadIdx.x;
  const int ch = vb0 + 16 * w + r16;  // the lane's value channel
  const bool on = ch < a.vd;

  // S[2 ks], S[2 ks + 1]: keys 32 ks + 8 g + 0..3, + 4..7 of the lane's channel
  f32x4_t S[KT];
  const int64_t state = (int64_t)a.vd * a.kd, seq_state = ((int64_t)seq * a.heads + head) * state;
  const uint32_t state_bytes = (uint32_t)state * 4;
  auto key_at = [&](int kt) { return 32 * (kt >> 1) + 8 * g + 4 * (kt & 1); };
  auto state_at = [&](int kt) {
    const int key = key_at(kt);
    return on && key < a.kd ? (uint32_t)(ch * a.kd + key) * 4 : 0x7f000000u;
  };
  {
    const float* from = BACK ? a.ds_last : a.s0;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(from ? from + seq_state : nullptr,
                                                from ? state_bytes : 0u);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      S[kt] = __builtin_bit_cast(f32x4_t,
                                 __builtin_amdgcn_raw_buffer_load_b128(rs, state_at(kt), 0, 0));
  }

  const IO* kp = static_cast<const IO*>(a.k.p) + (int64_t)(head / a.k.hdiv) * a.kd;
  const IO* qp = static_cast<const IO*>(a.q.p) + (int64_t)(head / a.q.hdiv) * a.kd;
  const DeltaOperand& vo = BACK ? a.dy : a.v;
  const IO* vp = static_cast<const IO*>(vo.p) + (int64_t)head * a.vd;
  const int64_t rec_size = delta_record(a.back);
  const int sides = a.back ? 2 : 1;

  Loader<IO, KD, THREADS> tk, tq;
  Loader<IO, VB, THREADS> tv;
  constexpr int kFragPasses = (kDeltaFrags + NW - 1) / NW;
  constexpr int kRowPasses = (kDeltaRows * C + 4 + THREADS * 4 - 1) / (THREADS * 4);
  Frag tf[kFragPasses];
  f32x4_t trow[kRowPasses];
  auto first_token = [&](int c) { return (int64_t)(s.first + c * C); };
  auto size = [&](int c) { return min(s.len - c * C, C); };
  auto record = [&](int c) { return a.record + ((int64_t)(s.chunk0 + c) * a.heads + head) * rec_size; };
  auto load = [&](int c) {
    const int n = size(c);
    const int64_t t0 = first_token(c);
    tk.load(kp + t0 * a.k.stride, a.k.stride, n, a.kd, 0, tid);
    if constexpr (W != kKeep) tq.load(qp + t0 * a.q.stride, a.q.stride, n, a.kd, 0, tid);
    tv.load(vp + t0 * vo.stride, vo.stride, n, a.vd, vb0, tid);
    const float* rec = record(c);
    const float* side = rec + (BACK ? kDeltaFrags * kDeltaFrag : 0);
#pragma unroll
    for (int p = 0; p < kFragPasses; ++p) {
      const int f = min(p * NW + w, kDeltaFrags - 1);
      const float* from = side + f * kDeltaFrag + lane * 8;
      tf[p] = Frag{*reinterpret_cast<const f32x4_t*>(from), *reinterpret_cast<const f32x4_t*>(from + 4)};
    }
    const float* rows = rec + sides * kDeltaFrags * kDeltaFrag;
#pragma unroll
    for (int p = 0; p < kRowPasses; ++p) {
      const int i = min((p * THREADS + tid) * 4, kDeltaRows * C);
      trow[p] = *reinterpret_cast<const f32x4_t*>(rows + i);
    }
  };

  if (threadIdx.x < 2) sh.odd[threadIdx.x] = 0;
  const int chunks = s.chunks;
  if (chunks > 0) load(BACK ? chunks - 1 : 0);
  lds_barrier();

  for (int step = 0; step < chunks; ++step) {
    const int c = BACK ? chunks - 1 - step : step, n = size(c);
    const int64_t t0 = first_token(c), unit = (int64_t)(s.chunk0 + c) * a.heads + head;
    // Addresses are derived from these anew in every chunk: kept over the loop
    // they would push the state out of the registers.
    asm volatile("" : "+v"(r16), "+v"(g), "+v"(tid));
    if (step > 0) lds_barrier();  // the previous chunk's tiles are read
    tk.store(sh.k, tid);
    if constexpr (W != kKeep) tq.store(sh.q, tid);
    tv.store(sh.v, tid);
#pragma unroll
    for (int p = 0; p < kFragPasses; ++p) {
      const int f = p * NW + w;
      if (f < kDeltaFrags) {
        const float x[8] = {tf[p].lo[0], tf[p].lo[1], tf[p].lo[2], tf[p].lo[3],
                            tf[p].hi[0], tf[p].hi[1], tf[p].hi[2], tf[p].hi[3]};
        M::template put<NP>(sh.t[f], lane, M::template split<NP>(x));
      }
    }
#pragma unroll
    for (int p = 0; p < kRowPasses; ++p) {
      const int i = (p * THREADS + tid) * 4;
      if (i < kDeltaRows * C) *reinterpret_cast<f32x4_t*>(&sh.rows[0][0] + i) = trow[p];
      if (i == kDeltaRows * C) *reinterpret_cast<f32x4_t*>(sh.ends) = trow[p];
    }
    const int parity = step & 1;
    if constexpr (!BACK) {
      if (tv.odd()) sh.odd[parity] = 1;
    }
    lds_barrier();
    if (step + 1 < chunks) load(BACK ? c - 1 : c + 1);
    const float dec = sh.ends[0], dec_low = sh.ends[1];
    bool odd = false;
    if constexpr (!BACK) {
      // A later token's infinity or NaN must not reach an earlier one through the
      // zeros of the triangles: such a chunk is walked token by token.
      odd = __builtin_amdgcn_readfirstlane((sh.ends[2] != 0.0f) | sh.odd[parity]) != 0;
    }
    if constexpr (W == kKeep) {
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.states + unit * state, state_bytes);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, S[kt]), rs, state_at(kt), 0,
                                               0);
    }
    if constexpr (BACK) {
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.adjoints + unit * state, state_bytes);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, S[kt]), rs, state_at(kt), 0,
                                               0);
    }

    if (!BACK && __builtin_expect(odd, 0)) {
      if constexpr (!BACK) {
        lds_barrier();  // as many as below
        if (threadIdx.x == 0) sh.odd[parity ^ 1] = 0;
        for (int t = 0; t < n; ++t) {
          float had = 0.0f, x[8], v = 0.0f;
          const float decay = sh.rows[kRowDecay][t];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            M::unpack(KTile::row8(sh.k, t, 32 * ks + 8 * g), x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (32 * ks + 8 * g < a.kd) {
                S[2 * ks + (j >> 2)][j & 3] *= decay;
                had = __builtin_fmaf(S[2 * ks + (j >> 2)][j & 3], x[j], had);
              }
            }
          }
          had += __shfl_xor(had, 16);
          had += __shfl_xor(had, 32);
          v = io<IO>::load(reinterpret_cast<const IO*>(sh.v + VTile::at(t, 16 * w + r16)));
          const float r = v - had, u = sh.rows[kRowBeta][t] * r;
          float dot = 0.0f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            float y[8];
            M::unpack(KTile::row8(sh.k, t, 32 * ks + 8 * g), x);
            if constexpr (W == kForward) M::unpack(KTile::row8(sh.q, t, 32 * ks + 8 * g), y);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (32 * ks + 8 * g < a.kd) {  // (no NaN in channels that there are not)
                const float z = __builtin_fmaf(u, x[j], S[2 * ks + (j >> 2)][j & 3]);
                S[2 * ks + (j >> 2)][j & 3] = z;
                if constexpr (W == kForward) dot = __builtin_fmaf(z, y[j], dot);
              }
            }
          }
          if constexpr (W == kForward) {
            dot += __shfl_xor(dot, 16);
            dot += __shfl_xor(dot, 32);
            if (on && g == 0)
              io<IO>::store(static_cast<IO*>(a.o) + ((t0 + t) * a.heads + head) * a.vd + ch,
                            dot * a.scale);
          } else if (on && g == 0) {
            a.r[(unit * C + t) * a.vd + ch] = r;
          }
        }
        if (W == kKeep && on && g == 0)
          for (int t = n; t < C; ++t) a.r[(unit * C + t) * a.vd + ch] = 0.0f;
        continue;
      }
    }

    // P, or its transpose, in fragments: of a tile of rows and 32 columns.
    // Forward: right operand, column t, slots s; back: left operand, row s, slots t.
    if constexpr (W != kKeep) {
#pragma unroll
      for (int p = 0; p < kFragPasses; ++p) {
        const int f = p * NW + w;
        if (f < kDeltaFrags) {
          const int tt = !BACK ? (f < 4 ? f : f - 2) : (f < 4 ? f >> 1 : f - 2);
          const int ks = !BACK ? (f < 4 ? 0 : 1) : (f < 4 ? f & 1 : 1);
          const int here = BACK ? row_of(tt, r16) : 16 * tt + r16;
          f32x4_t m[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
          const uint8_t *rt = BACK ? sh.q : sh.k, *ct = BACK ? sh.k : sh.q;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            const typename M::In col = KTile::row8(ct, here, 32 * kk + 8 * g);
#pragma unroll
            for (int half = 0; half < 2; ++half)
              m[half] = M::mm(KTile::row8(rt, row_of(2 * ks + half, r16), 32 * kk + 8 * g), col,
                              m[half]);
          }
          float x[8], gh[8], gl[8];
          rows8(sh.rows[kRowG], ks, g, gh);
          rows8(sh.rows[kRowGLow], ks, g, gl);
          const float hi = sh.rows[kRowG][here], lo = sh.rows[kRowGLow][here];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int other = 32 * ks + 8 * g + j;
            const float d = BACK ? (gh[j] - hi) + (gl[j] - lo) : (hi - gh[j]) + (lo - gl[j]);
            const bool pair = BACK ? other >= here : other <= here;
            x[j] = pair ? m[j >> 2][j & 3] * fast_exp2(d) * a.scale : 0.0f;
          }
          M::template put<kPP>(sh.p[f], lane, M::template split<kPP>(x));
        }
      }
    }

    // k S^T (rows: tokens), and q S^T the other way round (columns: tokens)
    f32x4_t x[4], o[W == kForward ? 4 : 1];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      x[tt] = f32x4_t{0, 0, 0, 0};
      if constexpr (W == kForward) o[tt] = x[tt];
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const float z[8] = {S[2 * ks][0], S[2 * ks][1], S[2 * ks][2], S[2 * ks][3],
                          S[2 * ks + 1][0], S[2 * ks + 1][1], S[2 * ks + 1][2], S[2 * ks + 1][3]};
      const auto sp = M::template split<NP>(z);
      typename M::In kr[4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) kr[tt] = KTile::row8(sh.k, row_of(tt, r16), 32 * ks + 8 * g);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) x[tt] = M::mm(kr[tt], sp, x[tt]);
      if constexpr (W == kForward) {
        const auto s2 = M::template first<2>(sp);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
          o[tt] = M::mm(s2, KTile::row8(sh.q, 16 * tt + r16, 32 * ks + 8 * g), o[tt]);
      }
    }

    // v or dy of the wave's channels: tokens 32 p + 8 g .. of channel r16
    typename M::In vc[2];
#pragma unroll
    for (int p = 0; p < 2; ++p)
      vc[p] = VTile::col8(sh.v, 32 * p + 8 * g, r16, [&](int i) { return 16 * w + i; });

    if constexpr (BACK) {
      lds_barrier();  // P is whole
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float gam[8];
        rows8(sh.rows[kRowGam], p, g, gam);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tt = 2 * p + h;
#pragma unroll
          for (int i = 0; i < 4; ++i) x[tt][i] *= gam[4 * h + i];
#pragma unroll
          for (int ks = p; ks < 2; ++ks)
            x[tt] = M::mm(M::template get<kPP>(sh.p[tt < 2 ? 2 * tt + ks : tt + 2], lane), vc[ks], x[tt]);
        }
      }
    } else {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float lam[8], v[8];
        rows8(sh.rows[kRowLam], p, g, lam);
        M::unpack(vc[p], v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[2 * p + (j >> 2)][j & 3] = __builtin_fmaf(-lam[j], x[2 * p + (j >> 2)][j & 3], v[j]);
      }
    }

    // the triangle's inverse
    f32x4_t r[4];
    {
      typename M::template Parts<NP> xp[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float z[8] = {x[2 * p][0], x[2 * p][1], x[2 * p][2], x[2 * p][3],
                            x[2 * p + 1][0], x[2 * p + 1][1], x[2 * p + 1][2], x[2 * p + 1][3]};
        xp[p] = M::template split<NP>(z);
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        r[tt] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int ks = BACK ? tt >> 1 : 0; ks < (BACK ? 2 : (tt >> 1) + 1); ++ks) {
          const int f = BACK ? (tt < 2 ? 2 * tt + ks : tt + 2) : (ks == 0 ? tt : tt + 2);
          r[tt] = M::mm(M::template get<NP>(sh.t[f], lane), xp[ks], r[tt]);
        }
      }
    }
    // r, or the adjoint of u, for the backward
    if constexpr (W != kForward) {
      const uint32_t row = (uint32_t)a.vd * 4;
      const __amdgpu_buffer_rsrc_t rs =
          make_rsrc((BACK ? a.y : a.r) + unit * C * a.vd, (uint32_t)C * row);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_buffer_store_b32(
              __float_as_uint(r[tt][i]), rs,
              on ? (uint32_t)row_of(tt, 4 * g + i) * row + (uint32_t)ch * 4 : 0x7f000000u, 0, 0);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float beta[8];
      rows8(sh.rows[kRowBeta], p, g, beta);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[2 * p + (j >> 2)][j & 3] *= beta[j];
    }
    if constexpr (BACK) {  // dv
      const uint32_t row = (uint32_t)a.heads * a.vd * (uint32_t)sizeof(IO);
      const __amdgpu_buffer_rsrc_t rs =
          make_rsrc(static_cast<IO*>(a.dv) + (t0 * a.heads + head) * a.vd,
                    (uint32_t)(n - 1) * row + (uint32_t)a.vd * (uint32_t)sizeof(IO));
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t to = on ? (uint32_t)row_of(tt, 4 * g + i) * row + (uint32_t)ch * (uint32_t)sizeof(IO)
                                 : 0x7f000000u;
          buf<IO>::store(r[tt][i], rs, to, 0);
        }
    }
    if constexpr (W == kForward) {
      lds_barrier();  // P is whole
      if (threadIdx.x == 0) sh.odd[parity ^ 1] = 0;
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) o[tt] *= sh.rows[kRowLam][16 * tt + r16] * a.scale;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float z[8] = {r[2 * p][0], r[2 * p][1], r[2 * p][2], r[2 * p][3],
                            r[2 * p + 1][0], r[2 * p + 1][1], r[2 * p + 1][2], r[2 * p + 1][3]};
        const auto up = M::template split<2>(z);
#pragma unroll
        for (int tt = 2 * p; tt < 4; ++tt)
          o[tt] = M::mm(up, M::template get<2>(sh.p[p == 0 ? tt : tt + 2], lane), o[tt]);
      }
      const int oc = vb0 + 16 * w + 4 * g;  // 4 channels of token 16 tt + r16
      const uint32_t row = (uint32_t)a.heads * a.vd * (uint32_t)sizeof(IO);
      const __amdgpu_buffer_rsrc_t rs =
          make_rsrc(static_cast<IO*>(a.o) + (t0 * a.heads + head) * a.vd,
                    (uint32_t)(n - 1) * row + (uint32_t)a.vd * (uint32_t)sizeof(IO));
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const uint32_t to = oc < a.vd ? (uint32_t)(16 * tt + r16) * row + (uint32_t)oc * (uint32_t)sizeof(IO)
                                      : 0x7f000000u;
        if constexpr (sizeof(IO) == 2)
          __builtin_amdgcn_raw_buffer_store_b64(to_bf16x4(o[tt]), rs, to, 0, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, o[tt]), rs, to, 0, 0);
      }
    }
    if constexpr (W == kKeep) {
      lds_barrier();  // as many as in a chunk walked token by token
      if (threadIdx.x == 0) sh.odd[parity ^ 1] = 0;
    }

    // the state: what the chunk adds is summed up first, its last parts first, and
    // the decay enters with what its fp32 number leaves of it, so that a state of
    // many chunks does not drift
    typename M::template Parts<NP> up[2], yp[BACK ? 2 : 1];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float z[8], wt[8];
      rows8(sh.rows[BACK ? kRowLam : kRowGam], p, g, wt);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        z[j] = r[2 * p + (j >> 2)][j & 3] * (BACK ? -wt[j] : wt[j]);
      up[p] = M::template split<NP>(z);
      if constexpr (BACK) {
        M::unpack(vc[p], z);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] *= wt[j] * a.scale;
        yp[p] = M::template split<NP>(z);
      }
    }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      // columns of the tile: keys 32 (kt / 2) + 8 (c / 4) + c % 4 (+ 4)
      auto keys = [&](int i) { return row_of(kt, i); };
      f32x4_t d{0, 0, 0, 0};
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        d = M::mm(KTile::col8(sh.k, 32 * p + 8 * g, r16, keys), up[p], d);
        if constexpr (BACK) d = M::mm(KTile::col8(sh.q, 32 * p + 8 * g, r16, keys), yp[p], d);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        S[kt][i] = __builtin_fmaf(dec, S[kt][i], __builtin_fmaf(dec_low, S[kt][i], d[i]));
    }
  }

  float* to = BACK ? a.ds0 : W == kForward ? a.s_last : nullptr;
  if (!to) return;
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(to + seq_state, state_bytes);
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, S[kt]), rs, state_at(kt), 0, 0);
}

// Blocks: sequences from the longest, heads, value blocks; the two walks of a
// backward side by side.
struct Grid {
  int64_t count;      // blocks of one walk
  uint32_t vblocks, group;
};

template <typename IO, int KD, int NW, Walk W>
__device__ __forceinline__ void walk_block(const DeltaArgs& a, const Grid& g, int64_t b, void* lds) {
  if (b >= g.count) return;
  const int64_t sh = b / g.vblocks;
  const int vb = (int)(b - sh * g.vblocks);
  int64_t seq = sh / a.heads;
  const int head = (int)(sh - seq * a.heads);
  if (a.cu) seq = a.table[a.nseq + 1 + seq];
  walk<IO, KD, NW, W>(a, *static_cast<Shared<IO, KD, NW, W>*>(lds), (int)seq, head, vb * 16 * NW);
}

template <typename IO, int KD, int NW>
__global__ __launch_bounds__(64 * NW) void delta_forward_kernel(DeltaArgs a, Grid g, int64_t block0) {
  __shared__ Shared<IO, KD, NW, kForward> sh;
  walk_block<IO, KD, NW, kForward>(a, g, block0 + xcd_block(blockIdx.x, g.group), &sh);
}
template <typename IO, int KD, int NW>
__global__ __launch_bounds__(64 * NW) void delta_backward_kernel(DeltaArgs a, Grid g, int64_t block0) {
  __shared__ union {
    Shared<IO, KD, NW, kKeep> keep;
    Shared<IO, KD, NW, kBack> back;
  } sh;
  const int64_t b = block0 + xcd_block(blockIdx.x, g.group);
  if (b & 1) walk_block<IO, KD, NW, kBack>(a, g, b >> 1, &sh);
  else walk_block<IO, KD, NW, kKeep>(a, g, b >> 1, &sh);
}

template <typename IO, int KD, int NW> hipError_t launch_nw(const DeltaArgs& a, hipStream_t stream) {
  Grid g;
  g.vblocks = (uint32_t)((a.vd + 16 * NW - 1) / (16 * NW));
  g.count = a.nseq * a.heads * g.vblocks;
  const int walks = a.back ? 2 : 1;
  g.group = std::min((uint32_t)a.rep * g.vblocks * walks, 4096u);
  const int64_t round = 8 * (int64_t)g.group, all = (g.count * walks + round - 1) / round * round;
  const int64_t most = max_blocks(64 * NW) / round * round;
  for (int64_t b = 0; b < all; b += most) {
    const dim3 grid((unsigned)std::min(all - b, most));
    if (a.back)
      hipLaunchKernelGGL((delta_backward_kernel<IO, KD, NW>), grid, dim3(64 * NW), 0, stream, a, g, b);
    else
      hipLaunchKernelGGL((delta_forward_kernel<IO, KD, NW>), grid, dim3(64 * NW), 0, stream, a, g, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Waves of a block.
inline int waves_of(const DeltaArgs& a) {
  return a.vd <= 16 ? 2 : a.vd <= 32 ? 2 : 4;
}

template <typename IO, int KD> hipError_t launch_kd(const DeltaArgs& a, hipStream_t stream) {
  switch (waves_of(a)) {
    case 2: return launch_nw<IO, KD, 2>(a, stream);
    default: return launch_nw<IO, KD, 4>(a, stream);
  }
}
template <typename IO> hipError_t launch_walk(const DeltaArgs& a, hipStream_t stream) {
  return a.kd <= 64 ? launch_kd<IO, 64>(a, stream) : launch_kd<IO, 128>(a, stream);
}

}  // namespace
}  // namespace ssm
