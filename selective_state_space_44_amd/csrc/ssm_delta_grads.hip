// ssm_delta_grads.hip -- the backward of the gated delta rule after its two walks
// (ssm_delta_walk.h): with the state S entering every chunk, the adjoint D leaving
// it, r and the adjoint y of u = b r, all chunks are independent (gfx950, wave64).
//
//   c_ts = scale exp(G_t - G_s) b_s (dy_t . r_s),            s <= t
//   m_ts = -exp(G_t - G_s) b_t b_s (y_t . r_s),               s < t
//   dq = scale exp(G) (dy S) + c k
//   dk = exp(G_end - G) b (r D) - exp(G) b (y S) + c^T q + (m + m^T) k
//   dbeta_t = y_t . r_t
// The decay of token i stands in every exp from before i to i or later, so its
// gradient is the sum of the terms that hold one:
//   dlog_decay_i = sum over s < i <= t of (c_ts q_t . k_s + m_ts k_t . k_s)
//     + sum over t >= i of exp(G_t) (scale (dy_t S) . q_t - b_t (y_t S) . k_t)
//     + sum over s < i of exp(G_end - G_s) b_s (r_s D) . k_s + exp(G_end) <D, S>.
// Each carries a_i itself: nothing is left of a decay of 0, nor at a first token that no
// state comes to, and little of a decay that leaves little.  (It is also a difference,
// of q . dq - v . dv summed from i on, but those sums hold what the decay cuts off: 1e-7
// of them stood where nothing is left, and 8.2e-7 of the whole over 100 tokens, 2.2e-7
// now, for 2% of a backward with heads of 128 and 5% of 64.)
//
// A block takes chunks of one key head, of each its value heads one after the other,
// and adds up their dq and dk in registers.  Each of its eight waves has 16 keys (of 64
// keys, and half of the tokens); r, y and dy go through LDS 64 value channels at a
// time, in bf16 parts, S and D straight into the registers of the one wave that has
// their keys, and all are asked for one step ahead, of the next chunk too: there is one
// block to a CU, held by its registers, and nothing else to wait beside: 8 x 2048 tokens
// of 24 heads of 64 275 us, 4 x 4096 of 40 over 8 of 128 790, 42% of the waves' cycles
// spent waiting (before dlog_decay's terms stood apart 251 and 723 on that card; on a
// quicker one 225, and 290 with a block to every chunk, and 725 both ways; with two sets
// of tiles in LDS and one barrier a step instead of two 311 and 718).  What dlog_decay
// (fp32) takes part in, and c on its way to dq, keeps three parts (24 bits), what else dq
// and dk (bf16) read two.
#include <algorithm>

#include "ssm_delta_mm.h"

namespace ssm {
namespace {

// [64, 64] computed values in LDS as N parts.
template <typename IO, int N> struct PartTile {
  typedef Mat<IO> M;
  typedef Tile<IO, 64> T;
  static constexpr int kN = sizeof(IO) == 2 ? N : 1, kBytes = kN * T::kBytes;
  __device__ __forceinline__ static void put8(uint8_t* t, int row, int col, const float* x) {
    const auto p = M::template split<N>(x);
    if constexpr (sizeof(IO) == 2) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        *reinterpret_cast<u32x4_t*>(t + i * T::kBytes + T::at(row, col)) = p.p[i];
    } else {
      *reinterpret_cast<f32x4_t*>(t + T::at(row, col)) = p.lo;
      *reinterpret_cast<f32x4_t*>(t + T::at(row, col + 4)) = p.hi;
    }
  }
  template <int K>
  __device__ __forceinline__ static typename M::template Parts<K> row8(const uint8_t* t, int row,
                                                                       int col) {
    typename M::template Parts<K> r;
    if constexpr (sizeof(IO) == 2) {
#pragma unroll
      for (int i = 0; i < K; ++i) r.p[i] = T::row8(t + i * T::kBytes, row, col);
    } else {
      const auto x = T::row8(t, row, col);
      r.lo = x.lo, r.hi = x.hi;
    }
    return r;
  }
  template <int K>
  __device__ __forceinline__ static typename M::template Parts<K> cols(const uint8_t* t, int p, int r16,
                                                                       int g, int col0) {
    typename M::template Parts<K> r;
    const int base = T::cols_base(r16, g, col0);
    if constexpr (sizeof(IO) == 2) {
#pragma unroll
      for (int i = 0; i < K; ++i) r.p[i] = T::cols(t + i * T::kBytes, base, p);
    } else {
      const auto x = T::cols(t, base, p);
      r.lo = x.lo, r.hi = x.hi;
    }
    return r;
  }
};

template <int CTRL> __device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// Sum over 8 consecutive lanes.
__device__ __forceinline__ float sum8(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  return v + dpp<0x141>(v);
}
__device__ __forceinline__ float sum16(float v) {
  v = sum8(v);
  return v + dpp<0x140>(v);  // mirrored halves
}
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float sum_groups(float v) {  // over the four lane groups
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

template <typename IO, int KD> struct alignas(256) GradShared {
  static constexpr int NW = 8, KG = KD / 16;
  uint8_t k[Tile<IO, KD>::kBytes], q[Tile<IO, KD>::kBytes];
  union {
    struct {
      uint8_t dy[Tile<IO, 64>::kBytes], r[PartTile<IO, 3>::kBytes], y[PartTile<IO, 3>::kBytes];
    };
    struct {
      uint8_t c[PartTile<IO, 3>::kBytes], m[PartTile<IO, 2>::kBytes];
    };
  };
  float rows[kDeltaRows][C];
  float ends[4];
  // dlog_decay's terms by token: of the states, and of the pairs, by the tile of t; of
  // those the sums over the s of the first half, by t of the second
  float in[KG][C], out[KG][C], across[4][C], half[C];
  float ds[NW];
};

template <typename IO, int KD>
__global__ __launch_bounds__(512) void delta_grads_kernel(DeltaArgs a) {
  typedef Mat<IO> M;
  typedef Tile<IO, KD> KTile;
  typedef Tile<IO, 64> VTile;
  typedef PartTile<IO, 3> P3;
  typedef PartTile<IO, 2> P2;
  constexpr int NW = 8, THREADS = 64 * NW, KG = KD / 16, TT = KG / 2;  // key groups, a wave's tiles
  __shared__ GradShared<IO, KD> sh;
  const int kheads = a.heads / a.rep;
  const int chunks = a.cu ? a.table[a.nseq] : (int)a.chunks;
  // A chunk of one key head, of n tokens from t0 on; beyond the last of none.
  struct Unit {
    int chunk, kh, t0, n;
  };
  auto unit_at = [&](int chunk, int kh) {
    Unit u{0, 0, 0, 0};
    if (chunk < chunks) {
      const Chunk c = chunk_of(a, chunk);
      u = Unit{chunk, kh, (int)c.t0, c.n};
    }
    return u;
  };
  Unit here = unit_at((int)blockIdx.x / kheads, (int)blockIdx.x % kheads);
  if (here.n == 0) return;
  const int w = wave_id();
  const int kg = w % KG, tt0 = w / KG * TT;
  int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
  // (Addresses are derived anew from the thread's number: kept, they would not fit.)
  auto anew = [&] {
    tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    lane = tid & 63, r16 = lane & 15, g = lane >> 4;
  };

  auto rows_of = [&](const DeltaOperand& o, const Unit& u, int head, int dim) {
    return static_cast<const IO*>(o.p) + u.t0 * o.stride + (int64_t)head * dim;
  };
  constexpr bool AHEAD = KD * sizeof(IO) <= 128;  // registers for the next keys and queries
  auto load_keys = [&](const Unit& u, auto& tk, auto& tq) {
    tk.load(rows_of(a.k, u, u.kh, a.kd), a.k.stride, u.n, a.kd, 0, tid);
    tq.load(rows_of(a.q, u, u.kh, a.kd), a.q.stride, u.n, a.kd, 0, tid);
  };
  Loader<IO, KD, THREADS> ahead_k, ahead_q;
  if constexpr (AHEAD) load_keys(here, ahead_k, ahead_q);

  // What comes from memory for 64 value channels of a head.
  const int64_t state = (int64_t)a.vd * a.kd;
  const uint32_t state_bytes = (uint32_t)state * 4, solve_bytes = (uint32_t)(C * a.vd) * 4;
  Loader<IO, 64, THREADS> tdy;
  f32x4_t rv[2], yv[2], trow;
  float S[2][8], D[2][8];
  auto load_rows = [&](const Unit& u, int head, int v0) {
    const int64_t unit = (int64_t)u.chunk * a.heads + head;
    tdy.load(rows_of(a.dy, u, head, a.vd), a.dy.stride, u.n, a.vd, v0, tid);
    const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.r + unit * C * a.vd, u.n ? solve_bytes : 0);
    const __amdgpu_buffer_rsrc_t ry = make_rsrc(a.y + unit * C * a.vd, u.n ? solve_bytes : 0);
    const int col = v0 + 8 * (tid & 7);  // 8 threads to a row
    const uint32_t at = col < a.vd ? (uint32_t)((tid >> 3) * a.vd + col) * 4 : 0x7f000000u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      rv[h] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rr, at + 16 * h, 0, 0));
      yv[h] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ry, at + 16 * h, 0, 0));
    }
    constexpr DeltaRecord R = delta_record(true);
    const float* rec = reinterpret_cast<const float*>(a.record + unit * R.size + R.rows);
    trow = f32x4_t{0, 0, 0, 0};
    if (tid < (kDeltaRows * C + 4) / 4) trow = *reinterpret_cast<const f32x4_t*>(rec + 4 * tid);
  };
  auto load_states = [&](const Unit& u, int head, int v0, int cs) {
    const int64_t unit = (int64_t)u.chunk * a.heads + head;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.states + unit * state, u.n ? state_bytes : 0);
    const __amdgpu_buffer_rsrc_t rd = make_rsrc(a.adjoints + unit * state, u.n ? state_bytes : 0);
    const int ch = v0 + 32 * cs + 8 * g, key = 16 * kg + r16;
    // (vdim is a multiple of 8)
    const uint32_t at = key < a.kd && ch < a.vd ? (uint32_t)(ch * a.kd + key) * 4 : 0x7f000000u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t to = at + (uint32_t)(j * a.kd) * 4;
      S[cs][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, to, 0, 0));
      D[cs][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rd, to, 0, 0));
    }
  };

  const f32x4_t none{0, 0, 0, 0};
  load_rows(here, here.kh * a.rep, 0);
  load_states(here, here.kh * a.rep, 0, 0);
  load_states(here, here.kh * a.rep, 0, 1);

  for (;;) {
    int chunk_then = here.chunk + (int)gridDim.x / kheads, kh_then = here.kh + (int)gridDim.x % kheads;
    if (kh_then >= kheads) kh_then -= kheads, ++chunk_then;
    const Unit then = unit_at(chunk_then, kh_then);
    const int64_t t0 = here.t0;
    const int kh = here.kh, n = here.n;
    anew();
    {  // (the last unit's are read)
      Loader<IO, KD, THREADS> tk, tq;
      if constexpr (AHEAD) tk = ahead_k, tq = ahead_q;
      else load_keys(here, tk, tq);
      tk.store(sh.k, tid);
      tq.store(sh.q, tid);
    }
    f32x4_t dq[TT], dk[TT];  // [token tile]: rows keys, column token
#pragma unroll
    for (int t = 0; t < TT; ++t) dq[t] = dk[t] = none;

    for (int vh = 0; vh < a.rep; ++vh) {
      const int head = kh * a.rep + vh;
      f32x4_t dys[TT], rds[TT], ys[TT];  // dy S, r D, y S
      f32x4_t pc[2], pm[2];              // c, m: the w-th fragment of the lower triangles
#pragma unroll
      for (int t = 0; t < TT; ++t) dys[t] = rds[t] = ys[t] = none;
      pc[0] = pc[1] = pm[0] = pm[1] = none;
      float ds = 0.0f, db = 0.0f;
      const FragAt fa = frag_at<false>(w);

      for (int v0 = 0; v0 < a.vd; v0 += 64) {
        // the next channels', of this head, of the next one or of the next unit's first
        const bool last = v0 + 64 >= a.vd, over = last && vh + 1 == a.rep;
        const Unit& next_unit = over ? then : here;
        const int next = last ? 0 : v0 + 64, next_head = over ? then.kh * a.rep : last ? head + 1 : head;
        anew();
        lds_barrier();  // what stood there is read
        if (v0 == 0) {
          if (4 * tid < kDeltaRows * C) *reinterpret_cast<f32x4_t*>(&sh.rows[0][0] + 4 * tid) = trow;
          else if (4 * tid == kDeltaRows * C) *reinterpret_cast<f32x4_t*>(sh.ends) = trow;
        }
        tdy.store(sh.dy, tid);
        {
          const int row = tid >> 3, col = 8 * (tid & 7);
          float r[8], y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = rv[j >> 2][j & 3], y[j] = yv[j >> 2][j & 3];
          P3::put8(sh.r, row, col, r);
          P3::put8(sh.y, row, col, y);
#pragma unroll
          for (int j = 0; j < 8; ++j) db = __builtin_fmaf(y[j], r[j], db);
        }
        load_rows(next_unit, next_head, next);
        lds_barrier();

#pragma unroll
        for (int cs = 0; cs < 2; ++cs) {
          anew();
          const int col = 32 * cs + 8 * g;
#pragma unroll
          for (int j = 0; j < 8; ++j) ds = __builtin_fmaf(S[cs][j], D[cs][j], ds);
          const auto sp = M::template split<3>(S[cs]), dp = M::template split<3>(D[cs]);
          load_states(next_unit, next_head, next, cs);
          // dy, r and y of the tokens, by their channels
#pragma unroll
          for (int half = 0; half < TT / 2; ++half) {
            typename M::In dyf[2];
            typename M::template Parts<3> rf[2], yf[2];
            f32x4_t x[2] = {dys[2 * half], dys[2 * half + 1]}, y[2] = {ys[2 * half], ys[2 * half + 1]},
                    z[2] = {rds[2 * half], rds[2 * half + 1]};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int row = 16 * (tt0 + 2 * half + t) + r16;
              dyf[t] = VTile::row8(sh.dy, row, col);
              rf[t] = P3::template row8<3>(sh.r, row, col);
              yf[t] = P3::template row8<3>(sh.y, row, col);
            }
            mm<M>(sp, dyf, x);
            mm<M>(dp, rf, z);
            mm<M>(sp, yf, y);
#pragma unroll
            for (int t = 0; t < 2; ++t)
              dys[2 * half + t] = x[t], rds[2 * half + t] = z[t], ys[2 * half + t] = y[t];
            __builtin_amdgcn_sched_barrier(0);
          }
          // pairs: tile tt of the tokens t against 32 of s
          if (w < kDeltaFrags) {
            const typename M::In dyw = VTile::row8(sh.dy, 16 * fa.tt + r16, col);
            const auto yw = P3::template row8<3>(sh.y, 16 * fa.tt + r16, col);
            typename M::template Parts<3> rw[2];
#pragma unroll
            for (int half = 0; half < 2; ++half)
              rw[half] = P3::template row8<3>(sh.r, row_of(2 * fa.ks + half, r16), col);
            mm<M>(rw, dyw, pc);
            mm<M>(rw, yw, pm);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }

      anew();
      lds_barrier();  // r, y and dy are read
      if (w < kDeltaFrags) {
        const int t = 16 * fa.tt + r16, s0 = 32 * fa.ks + 8 * g;
        f32x4_t qk[2] = {none, none}, kk[2] = {none, none};  // q_t . k_s, k_t . k_s
#pragma unroll
        for (int ks = 0; ks < KD / 32; ++ks) {
          typename M::In ka[2];
#pragma unroll
          for (int half = 0; half < 2; ++half)
            ka[half] = KTile::row8(sh.k, row_of(2 * fa.ks + half, r16), 32 * ks + 8 * g);
          mm<M>(ka, KTile::row8(sh.q, t, 32 * ks + 8 * g), qk);
          mm<M>(ka, KTile::row8(sh.k, t, 32 * ks + 8 * g), kk);
        }
        const float bt = sh.rows[kRowBeta][t], hi = sh.rows[kRowG][t], lo = sh.rows[kRowGLow][t];
        float c[8], m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int s = s0 + j;
          const float d = (hi - sh.rows[kRowG][s]) + (lo - sh.rows[kRowGLow][s]);
          const float wt = fast_exp2(d) * sh.rows[kRowBeta][s];
          c[j] = s <= t ? pc[j >> 2][j & 3] * wt * a.scale : 0.0f;
          m[j] = s < t ? -pm[j >> 2][j & 3] * wt * bt : 0.0f;
          qk[j >> 2][j & 3] = s < t ? c[j] * qk[j >> 2][j & 3] + m[j] * kk[j >> 2][j & 3] : 0.0f;
        }
        P3::put8(sh.c, t, s0, c);
        P2::put8(sh.m, t, s0, m);
        // Of token i, a source of the lane's: the pairs of t with the sources before i, in
        // this fragment, and of those the sum over the tile's t from i on.
        float before[8], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) before[j] = sum, sum += qk[j >> 2][j & 3];
        float upto = sum;
        {
          const float one = __shfl_up(upto, 16);
          upto += g >= 1 ? one : 0.0f;
          const float two = __shfl_up(upto, 32);
          upto += g >= 2 ? two : 0.0f;
        }
        if (fa.tt >= 2 && fa.ks == 0 && g == 3) sh.half[t] = upto;
        upto = __shfl_up(upto, 16);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float all = sum16(s0 + j <= t ? (g >= 1 ? upto : 0.0f) + before[j] : 0.0f);
          if (r16 == 0) sh.across[fa.tt][s0 + j] = all;
        }
      }
      {
        const int row = tid >> 3;
        const float d = sum8(db);
        if ((tid & 7) == 0 && row < n)
          io<IO>::store(static_cast<IO*>(a.dbeta) + (t0 + row) * a.heads + head, d);
      }
      lds_barrier();

      if constexpr (AHEAD)
        if (vh + 1 == a.rep) load_keys(then, ahead_k, ahead_q);
      // c k, c^T q, m k, m^T k, and what the states gave
      {
        typename M::In kc[2], qc[2];
        const int base = KTile::cols_base(r16, g, 16 * kg);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          kc[ks] = KTile::cols(sh.k, base, ks);
          qc[ks] = KTile::cols(sh.q, base, ks);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          anew();
          const int tt = tt0 + t, tok = 16 * tt + r16;
          const float lam = sh.rows[kRowLam][tok], beta = sh.rows[kRowBeta][tok];
          f32x4_t xk[1] = {none}, zk[1] = {none}, mk[1] = {none};
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            if (2 * ks <= tt) {  // sources s of the token
              const typename M::template Parts<3> cr[1] = {P3::template row8<3>(sh.c, tok, 32 * ks + 8 * g)};
              const typename M::template Parts<2> mr[1] = {P2::template row8<2>(sh.m, tok, 32 * ks + 8 * g)};
              mm<M>(kc[ks], cr, xk);
              mm<M>(kc[ks], mr, mk);
            }
            if (2 * ks + 1 >= tt) {  // tokens that read it
              const typename M::template Parts<2> cr[1] = {P3::template cols<2>(sh.c, ks, r16, g, 16 * tt)};
              const typename M::template Parts<2> mr[1] = {P2::template cols<2>(sh.m, ks, r16, g, 16 * tt)};
              mm<M>(qc[ks], cr, zk);
              mm<M>(kc[ks], mr, mk);
            }
          }
          const f32x4_t into = rds[t] * (sh.rows[kRowGam][tok] * beta);
          const f32x4_t of_q = dys[t] * (lam * a.scale), of_k = ys[t] * (lam * beta);
          dq[t] += of_q + xk[0];
          dk[t] += into - of_k + zk[0] + mk[0];
          // what the states gave, by q and k over the wave's keys, of which a lane has 4 g ..
          float in = 0.0f, out = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = KTile::at(tok, 16 * kg + 4 * g) + j * (int)sizeof(IO);
            const float kj = io<IO>::load(reinterpret_cast<const IO*>(sh.k + at));
            in = __builtin_fmaf(io<IO>::load(reinterpret_cast<const IO*>(sh.q + at)), of_q[j], in);
            in = __builtin_fmaf(-kj, of_k[j], in);
            out = __builtin_fmaf(kj, into[j], out);
          }
          in = sum_groups(in), out = sum_groups(out);
          if (g == 0) sh.in[kg][tok] = in, sh.out[kg][tok] = out;
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      anew();
      ds = sum64(ds);
      if (lane == 0) sh.ds[w] = tt0 == 0 ? ds : 0.0f;
      lds_barrier();
      if (w == 0) {
        double in = 0.0, out = 0.0, all = 0.0;
        float half = lane >= 32 ? sh.half[lane] : 0.0f, across = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) across += i >= 2 || lane < 32 ? sh.across[i][lane] : 0.0f;
#pragma unroll
        for (int i = 0; i < KG; ++i) in += (double)sh.in[i][lane], out += (double)sh.out[i][lane];
#pragma unroll
        for (int i = 0; i < NW; ++i) all += (double)sh.ds[i];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {  // sums over the tokens from each on, and up to it
          const double down = __shfl_down(in, d), up = __shfl_up(out, d);
          const float halves = __shfl_down(half, d);
          if (lane + d < 64) in += down, half += halves;
          if (lane >= d) out += up;
        }
        if (lane >= 32) across += half;
        out = __shfl_up(out, 1);  // before it
        if (lane == 0) out = 0.0;
        all *= (double)sh.ends[0] + (double)sh.ends[1];
        if (lane < n)
          a.dlog_decay[(t0 + lane) * a.heads + head] = (float)(((double)across + in) + (out + all));
      }
    }

#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int tok = 16 * (tt0 + t) + r16, first = 16 * kg + 4 * g;
      if (tok >= n || first >= a.kd) continue;
      const int64_t at = ((t0 + tok) * kheads + kh) * a.kd + first;
      IO *pq = static_cast<IO*>(a.dq) + at, *pk = static_cast<IO*>(a.dk) + at;
      if constexpr (sizeof(IO) == 2) {
        *reinterpret_cast<u32x2_t*>(pq) = to_bf16x4(dq[t]);
        *reinterpret_cast<u32x2_t*>(pk) = to_bf16x4(dk[t]);
      } else {
        *reinterpret_cast<f32x4_t*>(pq) = dq[t];
        *reinterpret_cast<f32x4_t*>(pk) = dk[t];
      }
    }
    if (then.n == 0) return;
    here = then;
  }
}

template <typename IO, int KD> hipError_t launch(const DeltaArgs& a, hipStream_t stream) {
  const int64_t blocks = std::min<int64_t>(a.chunks * (a.heads / a.rep), 256);
  hipLaunchKernelGGL((delta_grads_kernel<IO, KD>), dim3((unsigned)blocks), dim3(512), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grads(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  if (a.kd <= 64) return io_bf16 ? launch<bf16, 64>(a, stream) : launch<float, 64>(a, stream);
  return io_bf16 ? launch<bf16, 128>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace ssm
