// ssm_delta_walk.h -- the chunked walks of the gated delta rule (gfx950, wave64):
// included by ssm_delta_mm.hip (bf16) and ssm_delta_f32.hip.
//
// With the records of ssm_delta_prep.hip, a chunk of 64 tokens that the state S
// [vd, kd] enters is five products instead of 64 rank-one updates:
//   x = v - exp(G) (k S^T),   r = (1 + N b)^-1 x,   u = b r
//   o = scale exp(G) (q S^T) + P b r,    P_ts = scale exp(G_t - G_s) q_t . k_s, s <= t
//   S <- exp(G_end) S + sum over s of exp(G_end - G_s) u_s k_s^T.
// The backward walks twice: forward, without o, keeping the states S and r; and
// back with the adjoint D of the state,
//   du = exp(G_end - G) (k D^T) + P^T dy,   y = (1 + b N)^-T du,
//   dv = b y,   D <- exp(G_end) D + scale sum of exp(G) dy q^T - sum of exp(G) dv k^T,
// keeping D and y.  From those ssm_delta_grads.hip forms the other gradients, all
// chunks at once.
//
// A block of NW waves walks one sequence of one head over 16 NW value channels.
// Each wave owns 16 of them with their whole state in registers and everything
// computed from it: a result tile is, split into bf16 parts, the operand of the
// next product (ssm_delta_mm.h), so nothing of x, r, u or S is exchanged.  In LDS
// are the chunk's tiles of k, q and v, the inverse and P.  S and D, and what enters
// them, are sums of three parts (24 bits).  o is rounded to bf16 and P and u enter it
// as two.
//
// Bound by the vector units and the matrix cores, which hardly overlap, as the two waves
// of a SIMD go through the same phases at the same time (this schedule's doing, not the
// hardware's): a wave's chunk of 128 x 128 in bf16 is 182 matrix instructions of 16 cycles
// and some 900 vector ones of 4, most of them splits into parts; of the cycles of 4 x 4096
// tokens' walks of 40 heads 41% and 50%, 10 thousand a chunk for a wave alone, 13 for two
// on a SIMD.
#pragma once

#include <algorithm>

#include "ssm_delta_mm.h"

namespace ssm {
namespace {

// Outputs; states and r for a backward; its adjoint; of each the state alone.
enum Walk { kForward, kKeep, kBack, kForwardSpan, kKeepSpan, kBackSpan };
constexpr bool goes_back(Walk w) { return w == kBack || w == kBackSpan; }
constexpr bool reads_queries(Walk w) { return w == kForward || goes_back(w); }
constexpr bool is_span(Walk w) { return w >= kForwardSpan; }

// What a walk goes over: chunks [c0, c1) of its sequence, from a state and to one
// (null: zeros; not written).  A span's walk may take the unit matrix in and no
// values, kdim rows of it: what the chunks make of a state that enters them, which
// is written as the chunks' decay and the rest (delta_move_floats).
struct Span {
  int c0, c1;
  const float* from;
  float* to;
  bool unit;
};

__device__ __forceinline__ uint32_t xcd_block(uint32_t b, uint32_t group) {
  // Logical block number in a grid handed out round robin to the 8 XCDs: runs of
  // `group` blocks, which read the same keys, go to one XCD and share its L2.
  const uint32_t round = b / (8 * group), i = b - round * 8 * group;
  return round * 8 * group + (i & 7) * group + (i >> 3);
}

template <typename IO, int KD, int NW, Walk W> struct alignas(256) Shared {
  typedef Mat<IO> M;
  // fragments of the inverse, and of P b or P's transpose, in LDS
  static constexpr int VB = 16 * NW, kPP = goes_back(W) ? M::kParts : 2;
  static constexpr int kSolveFrag = M::template kFragBytes<M::kParts>;
  static constexpr int kPairFrag = M::template kFragBytes<kPP>;
  uint8_t k[Tile<IO, KD>::kBytes];
  uint8_t q[reads_queries(W) ? Tile<IO, KD>::kBytes : 16];
  uint8_t v[Tile<IO, VB>::kBytes];  // v or dy; then o
  uint8_t solve[kDeltaFrags * kSolveFrag];
  uint8_t pairs[reads_queries(W) ? kDeltaFrags * kPairFrag : 16];
  float rows[kDeltaRows][C];
  float ends[4];
  float odd[8];  // by wave: whether v holds an infinity or NaN
};

// Two chunks' tiles in LDS, where that leaves a block of 8 waves its CU: the next
// chunk's are written beside this one's products, and one barrier a chunk does
// instead of two, between which nothing is computed (4 x 4096 x 40 heads: 12.2
// thousand cycles a chunk with two).
template <typename IO, int KD, int NW, Walk W> constexpr bool twofold() {
  return NW == 8 && 2 * sizeof(Shared<IO, KD, NW, W>) <= 160 * 1024;
}
template <typename IO, int KD, int NW, Walk W> struct Tiles {
  Shared<IO, KD, NW, W> of[twofold<IO, KD, NW, W>() ? 2 : 1];
};

// The first and the last two of four.
template <typename T> __device__ __forceinline__ T (&head2(T (&x)[4]))[2] {
  return *reinterpret_cast<T(*)[2]>(x);
}
template <typename T> __device__ __forceinline__ T (&tail2(T (&x)[4]))[2] {
  return *reinterpret_cast<T(*)[2]>(x + 2);
}

// 8 values by token 32 p + 8 g ..
__device__ __forceinline__ void rows8(const float* row, int p, int g, float* x) {
  const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(row + 32 * p + 8 * g);
  const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(row + 32 * p + 8 * g + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = lo[i], x[4 + i] = hi[i];
}

template <typename IO, int KD, int NW, Walk W>
__device__ __forceinline__ void walk(const DeltaArgs& a, Tiles<IO, KD, NW, W>& tiles, int seq,
                                     int head, int vb0, const Span& span) {
  typedef Mat<IO> M;
  constexpr int VB = 16 * NW, THREADS = 64 * NW, KT = KD / 16, KS = KD / 32, NP = M::kParts;
  typedef Tile<IO, KD> KTile;
  typedef Tile<IO, VB> VTile;
  constexpr bool BACK = goes_back(W);
  Seq s = seq_of(a, seq);
  s.first += span.c0 * C;
  s.chunk0 += span.c0;
  s.chunks = min(s.chunks, span.c1) - span.c0;
  s.len = min(s.len - span.c0 * C, s.chunks * C);
  const bool unit_in = is_span(W) && span.unit;
  const int w = wave_id(), lane = threadIdx.x & 63;
  int r16 = lane & 15, g = lane >> 4, tid = threadIdx.x;
  const int ch = vb0 + 16 * w + r16;  // the lane's value channel
  const int channels = unit_in ? a.kd : a.vd;
  const bool on = ch < channels;

  // S[2 ks], S[2 ks + 1]: keys 32 ks + 8 g + 0..3, + 4..7 of the lane's channel
  f32x4_t S[KT];
  const int64_t state = (int64_t)a.vd * a.kd;
  const uint32_t state_bytes = (uint32_t)(channels * a.kd) * 4;
  auto key_at = [&](int kt) { return 32 * (kt >> 1) + 8 * g + 4 * (kt & 1); };
  auto state_at = [&](int kt) {
    const int key = key_at(kt);
    return on && key < a.kd ? (uint32_t)(ch * a.kd + key) * 4 : 0x7f000000u;
  };
  {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(span.from, span.from ? state_bytes : 0u);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      S[kt] = __builtin_bit_cast(f32x4_t,
                                 __builtin_amdgcn_raw_buffer_load_b128(rs, state_at(kt), 0, 0));
  }
  // Of the unit matrix S is what the chunks added: it enters them as S + decay 1, whose
  // decay is kept in 64 bits.  k (S + decay 1)^T is k S^T + decay k: the keys of the lane's
  // channel stand in v's place.
  double decay = unit_in ? 1.0 : 0.0;
  auto on_diagonal = [&](float add) {
    if constexpr (is_span(W) && !BACK) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (key_at(kt) + i == ch) S[kt][i] += add;
    }
  };

  const IO* kp = static_cast<const IO*>(a.k.p) + (int64_t)(head / a.k.hdiv) * a.kd;
  const IO* qp = static_cast<const IO*>(a.q.p) + (int64_t)(head / a.q.hdiv) * a.kd;
  const DeltaOperand& vo = BACK ? a.dy : a.v;
  const IO* vp = static_cast<const IO*>(vo.p) + (int64_t)head * a.vd;
  constexpr DeltaRecord R = delta_record(W != kForward && W != kForwardSpan);
  typedef Shared<IO, KD, NW, W> Sh;
  constexpr bool TWO = twofold<IO, KD, NW, W>();
  constexpr bool PAIR_PARTS = W == kForward && sizeof(IO) == 2;  // P b stands in parts

  Loader<IO, KD, THREADS> tk, tq;
  Loader<IO, VB, THREADS> tv;
  // fragments: the inverse's, then P's where it is to be split, by waves; P's in
  // parts, and the rows, in pieces
  constexpr int kSplit = !reads_queries(W) || PAIR_PARTS ? kDeltaFrags : 2 * kDeltaFrags;
  constexpr int kFragPasses = (kSplit + NW - 1) / NW;
  constexpr int kPieces = PAIR_PARTS ? kDeltaFrags * kDeltaFragBytes / 16 : 0;
  constexpr int kPiecePasses = (kPieces + THREADS - 1) / THREADS;
  constexpr int kRowPieces = kDeltaRows * C / 4 + 1;
  constexpr int kRowPasses = (kRowPieces + THREADS - 1) / THREADS;
  f32x4_t tf[kFragPasses][2];
  u32x4_t tp[kPiecePasses ? kPiecePasses : 1], trow[kRowPasses];
  const int chunks = s.chunks;
  // Loads past the last chunk, and the leaving of an o before the first, are made
  // all the same, over no memory: with as many accesses in every chunk the waits
  // are for the right ones.
  auto chunk_at = [&](int step) { return BACK ? chunks - 1 - step : step; };
  auto first_token = [&](int c) { return (int64_t)(s.first + max(c, 0) * C); };
  auto size = [&](int c) { return c >= 0 && c < chunks ? min(s.len - c * C, C) : 0; };
  auto load_k = [&](int c) {
    tk.load(kp + first_token(c) * a.k.stride, a.k.stride, size(c), a.kd, 0, tid);
  };
  auto load_q = [&](int c) {
    if constexpr (reads_queries(W))
      tq.load(qp + first_token(c) * a.q.stride, a.q.stride, size(c), a.kd, 0, tid);
  };
  auto load_v = [&](int c) {
    const IO* p = unit_in ? kp + first_token(c) * a.k.stride : vp + first_token(c) * vo.stride;
    tv.load(p, unit_in ? a.k.stride : vo.stride, size(c), channels, vb0, tid);
  };
  auto record = [&](int c) {
    return make_rsrc(a.record + ((int64_t)(s.chunk0 + max(c, 0)) * a.heads + head) * R.size,
                     c >= 0 && c < chunks ? R.size : 0);
  };
  auto load_frags = [&](int c) {
    const __amdgpu_buffer_rsrc_t rs = record(c);
#pragma unroll
    for (int p = 0; p < kFragPasses; ++p) {
      // (the last waves' may be none: over no memory)
      const int f = p * NW + w;
      const uint32_t at = (BACK ? (f < kDeltaFrags ? R.back : R.pairs - kDeltaFrags * kDeltaFragBytes)
                                : R.solve) + f * kDeltaFragBytes + lane * 16;
      const uint32_t from = f < kSplit ? at : 0x7f000000u;
      tf[p][0] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, from, 0, 0));
      tf[p][1] =
          __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, from + 1024, 0, 0));
    }
  };
  auto load_pieces = [&](int c) {
    const __amdgpu_buffer_rsrc_t rs = record(c);
#pragma unroll
    for (int p = 0; p < kPiecePasses; ++p) {
      const int i = p * THREADS + tid;
      tp[p] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                              rs, i < kPieces ? R.pairs + i * 16 : 0x7f000000u, 0, 0));
    }
#pragma unroll
    for (int p = 0; p < kRowPasses; ++p) {
      const int i = p * THREADS + tid;
      trow[p] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                       rs, i < kRowPieces ? R.rows + i * 16 : 0x7f000000u, 0, 0));
    }
  };
  auto store_k = [&](Sh& sh) { tk.store(sh.k, tid); };
  auto store_q = [&](Sh& sh) {
    if constexpr (reads_queries(W)) tq.store(sh.q, tid);
  };
  auto store_frags = [&](Sh& sh) {
#pragma unroll
    for (int p = 0; p < kFragPasses; ++p) {
      const int f = p * NW + w;
      if (f < kSplit) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = tf[p][j >> 2][j & 3];
        if (f < kDeltaFrags)
          M::template put<NP>(sh.solve + f * Sh::kSolveFrag, lane, M::template split<NP>(x));
        else
          M::template put<Sh::kPP>(sh.pairs + (f - kDeltaFrags) * Sh::kPairFrag, lane,
                                   M::template split<Sh::kPP>(x));
      }
    }
  };
  auto store_pieces = [&](Sh& sh) {
#pragma unroll
    for (int p = 0; p < kPiecePasses; ++p)
      if (p * THREADS + tid < kPieces)
        *reinterpret_cast<u32x4_t*>(sh.pairs + (p * THREADS + tid) * 16) = tp[p];
#pragma unroll
    for (int p = 0; p < kRowPasses; ++p)
      if (p * THREADS + tid < kRowPieces)
        *reinterpret_cast<u32x4_t*>(&sh.rows[0][0] + (p * THREADS + tid) * 4) = trow[p];
  };
  // A chunk's o stands in v's tile when the chunk is done, each wave's in the channels
  // that it alone read, and leaves from there in whole rows.  A thread takes exactly
  // the pieces that it fills with the next tile there.
  auto leave = [&](int c, Sh& sh, const Loader<IO, VB, THREADS>* then) {
    typedef Loader<IO, VB, THREADS> L;
    const uint32_t row = (uint32_t)a.heads * a.vd * (uint32_t)sizeof(IO);
    const int n = size(c);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(
        static_cast<IO*>(a.o) + (first_token(c) * a.heads + head) * a.vd,
        n > 0 ? (uint32_t)(n - 1) * row + (uint32_t)a.vd * (uint32_t)sizeof(IO) : 0u);
    u32x4_t o[L::kPasses];
#pragma unroll
    for (int p = 0; p < L::kPasses; ++p)
      if (L::kAll || L::row(p, tid) < C)
        o[p] = *reinterpret_cast<const u32x4_t*>(sh.v + L::slot(L::slot_base(tid), p));
    if (then) then->store(sh.v, tid);
    const int to = vb0 + L::col(0, tid);
    const uint32_t at = to < a.vd ? (uint32_t)L::row(0, tid) * row + (uint32_t)to * (uint32_t)sizeof(IO)
                                  : 0x7f000000u;
#pragma unroll
    for (int p = 0; p < L::kPasses; ++p)
      if (L::kAll || L::row(p, tid) < C)
        __builtin_amdgcn_raw_buffer_store_b128(o[p], rs, at + (uint32_t)(p * L::kRows) * row, 0, 0);
  };
  // v of the next chunk in; the o of chunk `out` out
  auto store_v = [&](Sh& sh, int out) {
    if constexpr (!BACK) {
      const bool odd = __ballot(tv.odd()) != 0;
      if (lane == 0) sh.odd[w] = odd ? 1.0f : 0.0f;
    }
    if constexpr (W == kForward) leave(out, sh, &tv);
    else tv.store(sh.v, tid);
  };
  auto load = [&](int c) {
    load_k(c);
    load_q(c);
    load_frags(c);
    load_pieces(c);
    load_v(c);
  };
  // (v last: waits for loads after o's stores would be for those as well)
  auto store = [&](Sh& sh, int out) {
    store_k(sh);
    store_q(sh);
    store_frags(sh);
    store_pieces(sh);
    store_v(sh, out);
  };
  if (chunks > 0) load(chunk_at(0));
  // (waited for here: a wait in the loop would be for its stores as well)
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) asm volatile("" : "+v"(S[kt]));
  if (TWO && chunks > 0) {
    store(tiles.of[0], -1);
    load(chunk_at(1));
    lds_barrier();
  }

  for (int step = 0; step < chunks; ++step) {
    const int c = chunk_at(step), n = size(c);
    const int64_t t0 = first_token(c), unit = (int64_t)(s.chunk0 + c) * a.heads + head;
    // Addresses are derived from these anew in every chunk: kept over the loop
    // they would push the state out of the registers.
    asm volatile("" : "+v"(r16), "+v"(g), "+v"(tid));
    Sh& sh = tiles.of[TWO ? step & 1 : 0];
    if constexpr (!TWO) {
      if (step > 0) lds_barrier();  // the previous chunk's tiles are read
      store(sh, step > 0 ? c - 1 : -1);
      lds_barrier();
    }
    // Beside this chunk's products the next one's tiles go into LDS, and those after
    // are asked for, a few at a time: all at once they would hold the waves up at
    // the memory pipe.  In order: keys, queries, fragments, pieces, v.
    Sh& other = tiles.of[TWO ? ~step & 1 : 0];
    const int ask = chunk_at(step + (TWO ? 2 : 1));
    auto advance = [&](int part) {
      if constexpr (TWO) {
        if (part == 0) store_k(other);
        if (part == 1) store_q(other);
        if (part == 2) store_frags(other);
        if (part == 3) store_pieces(other);
        if (part == 4) store_v(other, c - 1);
      }
      if (part == 0) load_k(ask);
      if (part == 1) load_q(ask);
      if (part == 2) load_frags(ask);
      if (part == 3) load_pieces(ask);
      if (part == 4) load_v(ask);
    };
    const float dec = sh.ends[0], dec_low = sh.ends[1];
    bool odd = false;
    if constexpr (!BACK) {
      // A later token's infinity or NaN must not reach an earlier one through the
      // zeros of the triangles: such a chunk is walked token by token.
      float any = sh.ends[2];
#pragma unroll
      for (int i = 0; i < NW; ++i) any += sh.odd[i];
      odd = __builtin_amdgcn_readfirstlane(any != 0.0f) != 0;
    }
    if constexpr (W == kKeep) {
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.states + unit * state, state_bytes);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, S[kt]), rs, state_at(kt), 0,
                                               0);
    }
    if constexpr (W == kBack) {
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.adjoints + unit * state, state_bytes);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, S[kt]), rs, state_at(kt), 0,
                                               0);
    }

    if (!BACK && __builtin_expect(odd, 0)) {
      if constexpr (!BACK) {
#pragma unroll
        for (int i = 0; i < 5; ++i) advance(i);
        if (unit_in) on_diagonal((float)decay);
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
          const float r = (unit_in ? 0.0f : v) - had, u = sh.rows[kRowBeta][t] * r;
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
            if (g == 0)
              io<IO>::store(reinterpret_cast<IO*>(sh.v + VTile::at(t, 16 * w + r16)), dot * a.scale);
          } else if (W == kKeep && on && g == 0) {
            a.r[(unit * C + t) * a.vd + ch] = r;
          }
        }
        if (W == kKeep && on && g == 0)
          for (int t = n; t < C; ++t) a.r[(unit * C + t) * a.vd + ch] = 0.0f;
        if (unit_in) {
          decay *= (double)dec + (double)dec_low;
          on_diagonal(-(float)decay);
          on_diagonal(-(float)(decay - (double)(float)decay));
        }
        if constexpr (TWO) lds_barrier();
        continue;
      }
    }

    // k S^T (rows: tokens), and q S^T the other way round (columns: tokens)
    const int row_at = KTile::rows_base(r16, g);
    f32x4_t x[4], o[W == kForward ? 4 : 1];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      x[tt] = f32x4_t{0, 0, 0, 0};
      if constexpr (W == kForward) o[tt] = x[tt];
    }
    // (the operands of the next 32 keys are read and split between the products of
    // these: a matrix instruction leaves time for three others)
    typename M::In kr[2][4], qr[W == kForward ? 2 : 1][4];
    typename M::template Parts<NP> sp[2];
    auto operands = [&](int ks) {
      const float z[8] = {S[2 * ks][0], S[2 * ks][1], S[2 * ks][2], S[2 * ks][3],
                          S[2 * ks + 1][0], S[2 * ks + 1][1], S[2 * ks + 1][2], S[2 * ks + 1][3]};
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        kr[ks & 1][tt] = KTile::rows(sh.k, row_at, tt, ks);
        if constexpr (W == kForward) qr[ks & 1][tt] = KTile::rows(sh.q, row_at, tt, ks);
      }
      sp[ks & 1] = M::template split<NP>(z);
    };
    operands(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks + 1 < KS) operands(ks + 1);
      if (ks == 0) advance(0);
      if (ks == KS / 2) advance(1);
      mm<M>(kr[ks & 1], sp[ks & 1], x);
      if constexpr (W == kForward) mm<M>(M::template first<2>(sp[ks & 1]), qr[ks & 1], o);
      if (sizeof(IO) == 2) {
#pragma unroll
        for (int i = 0; i < (W == kForward ? 20 : 12); ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix
          if (i < (W == kForward ? 8 : 4)) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS reads
          __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);  // vector
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }

    // v or dy of the wave's channels: tokens 32 p + 8 g .. of channel r16
    typename M::In vc[2];
#pragma unroll
    for (int p = 0; p < 2; ++p)
      vc[p] = VTile::cols(sh.v, VTile::cols_base(r16, g, 16 * w), p);

    auto solve_frag = [&](int f) {
      return M::template get<NP>(sh.solve + f * Sh::kSolveFrag, lane);
    };
    auto pair_frag = [&](int f) {
      return M::template get<Sh::kPP>(sh.pairs + f * Sh::kPairFrag, lane);
    };
    advance(2);
    if constexpr (BACK) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float gam[8];
        rows8(sh.rows[kRowGam], p, g, gam);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[2 * p + (j >> 2)][j & 3] *= gam[j];
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {  // rows up to the 32 columns'
        typename M::template Parts<Sh::kPP> pf[4];
#pragma unroll
        for (int tt = 0; tt < 2 * ks + 2; ++tt) pf[tt] = pair_frag(frag_of<true>(tt, ks));
        if (ks == 0) mm<M>(head2(pf), vc[ks], head2(x));
        else mm<M>(pf, vc[ks], x);
      }
    } else {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float lam[8], v[8];
        rows8(sh.rows[kRowLam], p, g, lam);
        M::unpack(vc[p], v);
        if constexpr (is_span(W)) {
          const float keys = (float)decay, values = unit_in ? 0.0f : 1.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[2 * p + (j >> 2)][j & 3] = __builtin_fmaf(keys, v[j], x[2 * p + (j >> 2)][j & 3]);
            v[j] *= values;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[2 * p + (j >> 2)][j & 3] = __builtin_fmaf(-lam[j], x[2 * p + (j >> 2)][j & 3], v[j]);
      }
    }

    __builtin_amdgcn_sched_barrier(0);
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
      for (int tt = 0; tt < 4; ++tt) r[tt] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        typename M::template Parts<NP> tf_[4];
#pragma unroll
        for (int tt = BACK ? 0 : 2 * ks; tt < (BACK ? 2 * ks + 2 : 4); ++tt)
          tf_[tt] = solve_frag(frag_of<BACK>(tt, ks));
        if (ks == (BACK ? 1 : 0)) mm<M>(tf_, xp[ks], r);
        else if (BACK) mm<M>(head2(tf_), xp[ks], head2(r));
        else mm<M>(tail2(tf_), xp[ks], tail2(r));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    advance(3);
    // r, or the adjoint of u, for the backward
    if constexpr (W == kKeep || W == kBack) {
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
    if constexpr (BACK) {  // dv
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float beta[8];
        rows8(sh.rows[kRowBeta], p, g, beta);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[2 * p + (j >> 2)][j & 3] *= beta[j];
      }
    }
    if constexpr (W == kBack) {
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
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) o[tt] *= sh.rows[kRowLam][row_of(tt, r16)] * a.scale;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float z[8] = {r[2 * p][0], r[2 * p][1], r[2 * p][2], r[2 * p][3],
                            r[2 * p + 1][0], r[2 * p + 1][1], r[2 * p + 1][2], r[2 * p + 1][3]};
        const auto up = M::template split<2>(z);
        typename M::template Parts<2> pf[4];
#pragma unroll
        for (int tt = 2 * p; tt < 4; ++tt) pf[tt] = pair_frag(frag_of<false>(tt, p));
        if (p == 0) mm<M>(up, pf, o);
        else mm<M>(up, tail2(pf), tail2(o));
      }
      // 4 channels of a token
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        uint8_t* to = sh.v + VTile::shift(VTile::at(row_of(0, r16), 16 * w + 4 * g),
                                          32 * (tt >> 1) + 4 * (tt & 1), 0);
        if constexpr (sizeof(IO) == 2) *reinterpret_cast<u32x2_t*>(to) = to_bf16x4(o[tt]);
        else *reinterpret_cast<f32x4_t*>(to) = o[tt];
      }
    }

    __builtin_amdgcn_sched_barrier(0);
    advance(4);
    // the state: what the chunk adds is summed up first, its last parts first, and
    // the decay enters with what its fp32 number leaves of it, so that a state of
    // many chunks does not drift
    typename M::template Parts<NP> up[2], yp[BACK ? 2 : 1];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float z[8], wt[8], beta[8];
      rows8(sh.rows[BACK ? kRowLam : kRowGam], p, g, wt);
      if constexpr (!BACK) rows8(sh.rows[kRowBeta], p, g, beta);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        z[j] = r[2 * p + (j >> 2)][j & 3] * (BACK ? -wt[j] : wt[j] * beta[j]);
      up[p] = M::template split<NP>(z);
      if constexpr (BACK) {
        M::unpack(vc[p], z);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] *= wt[j] * a.scale;
        yp[p] = M::template split<NP>(z);
      }
    }
    const int key_base = KTile::keys_base(r16, g);
#pragma unroll
    for (int k0 = 0; k0 < KT; k0 += 4) {
      f32x4_t d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        typename M::In kc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kc[i] = KTile::cols(sh.k, key_base, p, k0 + i);
        mm<M>(kc, up[p], d);
        if constexpr (BACK) {
#pragma unroll
          for (int i = 0; i < 4; ++i) kc[i] = KTile::cols(sh.q, key_base, p, k0 + i);
          mm<M>(kc, yp[p], d);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          S[k0 + i][j] = __builtin_fmaf(dec, S[k0 + i][j], __builtin_fmaf(dec_low, S[k0 + i][j], d[i][j]));
    }
    if (unit_in) decay *= (double)dec + (double)dec_low;
    if constexpr (TWO) lds_barrier();  // this chunk's tiles are read, the next one's whole
  }

  if (W == kForward && chunks > 0) {
    if constexpr (!TWO) lds_barrier();
    leave(chunks - 1, tiles.of[TWO ? (chunks - 1) & 1 : 0], nullptr);
  }
  if (!span.to) return;
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(span.to, state_bytes);
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, S[kt]), rs, state_at(kt), 0, 0);
  if (unit_in && vb0 == 0 && tid == 0) {
    float* to = span.to + (int64_t)a.kd * a.kd;
    to[0] = (float)decay;
    to[1] = (float)(decay - (double)to[0]);
  }
}

// Blocks: sequences from the longest, heads, value blocks; the two walks of a
// backward side by side.
struct Grid {
  int64_t count;      // blocks of one walk
  uint32_t vblocks, group;
};

__device__ __forceinline__ float* state_of(float* all, const DeltaArgs& a, int64_t unit) {
  return all ? all + unit * ((int64_t)a.vd * a.kd) : nullptr;
}
__device__ __forceinline__ const float* state_of(const float* all, const DeltaArgs& a, int64_t unit) {
  return state_of(const_cast<float*>(all), a, unit);
}

template <typename IO, int KD, int NW, Walk W>
__device__ __forceinline__ void walk_block(const DeltaArgs& a, const Grid& g, int64_t b, void* lds) {
  if (b >= g.count) return;
  const int64_t sh = b / g.vblocks;
  const int vb = (int)(b - sh * g.vblocks);
  int64_t seq = sh / a.heads;
  const int head = (int)(sh - seq * a.heads);
  if (a.cu) seq = a.table[a.nseq + 1 + seq];
  const int64_t unit = seq * a.heads + head;
  const Span span{0, INT32_MAX, state_of(W == kBack ? a.ds_last : a.s0, a, unit),
                  state_of(W == kBack ? a.ds0 : W == kForward ? a.s_last : nullptr, a, unit), false};
  walk<IO, KD, NW, W>(a, *static_cast<Tiles<IO, KD, NW, W>*>(lds), (int)seq, head, vb * 16 * NW, span);
}

// Blocks of four waves that a CU has LDS for.
template <typename IO, int KD, int NW> constexpr int blocks_of() {
  return NW == 4 && 2 * std::max(sizeof(Tiles<IO, KD, NW, kForward>), sizeof(Tiles<IO, KD, NW, kBack>)) <=
                        160 * 1024
             ? 2
             : 1;
}

template <typename IO, int KD, int NW>
__global__ __launch_bounds__(64 * NW, (blocks_of<IO, KD, NW>())) void delta_forward_kernel(
    DeltaArgs a, Grid g, int64_t block0) {
  __shared__ Tiles<IO, KD, NW, kForward> sh;
  walk_block<IO, KD, NW, kForward>(a, g, block0 + xcd_block(blockIdx.x, g.group), &sh);
}
template <typename IO, int KD, int NW>
__global__ __launch_bounds__(64 * NW, (blocks_of<IO, KD, NW>())) void delta_backward_kernel(
    DeltaArgs a, Grid g, int64_t block0) {
  __shared__ union {
    Tiles<IO, KD, NW, kKeep> keep;
    Tiles<IO, KD, NW, kBack> back;
  } sh;
  const int64_t b = block0 + xcd_block(blockIdx.x, g.group);
  if (b & 1) walk_block<IO, KD, NW, kBack>(a, g, b >> 1, &sh);
  else walk_block<IO, KD, NW, kKeep>(a, g, b >> 1, &sh);
}

// Few sequences and heads leave most CUs without a block.  The state after a span of
// chunks is E = L + S W, with L what a zero state becomes and W what the rows of a
// unit matrix become without values (kept as its decay and the rest), so the spans of a sequence are walked at the
// same time: the first as it is and of the others up to the last but one L and W;
// then their states are taken from one to the next (ssm_delta_spans.hip); and the
// second to the last are walked once more, as they are.  The adjoint goes through the
// spans the other way, by the same W transposed.
template <typename IO, int KD, int NW, bool BACK>
__global__ __launch_bounds__(64 * NW, (blocks_of<IO, KD, NW>())) void delta_spans_kernel(
    DeltaArgs a, uint32_t vblocks, uint32_t kblocks, int second) {
  constexpr Walk kWhole = BACK ? kKeep : kForward, kPart = BACK ? kKeepSpan : kForwardSpan;
  __shared__ union {
    Tiles<IO, KD, NW, kWhole> whole;
    Tiles<IO, KD, NW, kPart> part;
    Tiles<IO, KD, NW, BACK ? kBack : kPart> back;
    Tiles<IO, KD, NW, BACK ? kBackSpan : kPart> back_part;
  } sh;
  // Blocks: all spans' walks, the adjoint's, in the first launch the W's; spans, heads.
  // (Runs of a kind, so that those with nothing to do are spread over the XCDs: a span's
  // walk and W side by side left every second one the half of the work, 32 against 25 us
  // at 3 x 517 tokens.)
  const uint32_t walks = (uint32_t)a.spans * (uint32_t)a.heads * vblocks;
  const bool adjoint = BACK && blockIdx.x >= walks && blockIdx.x < 2 * walks;
  const bool moved = blockIdx.x >= walks && !adjoint;
  const uint32_t job = blockIdx.x - (moved ? (BACK ? 2 : 1) * walks : adjoint ? walks : 0);
  const uint32_t blocks = moved ? kblocks : vblocks, unit = job / blocks;
  const int vb0 = (int)(job - unit * blocks) * 16 * NW;
  const int head = (int)(unit % (uint32_t)a.heads);
  const SpanAt at = span_at(a, (int)(unit / (uint32_t)a.heads));
  if (at.seq < 0) return;
  const int j = at.j, last = at.n - 1;
  // Of this span and head, a sequence's last has none; those of the span before are so
  // much further up.
  const int64_t state = (int64_t)a.vd * a.kd, move = delta_move_floats(a.kd), before = a.heads * state;
  const int64_t seq_head = (int64_t)at.seq * a.heads + head;
  const int64_t kept = (int64_t)unit - (int64_t)at.seq * a.heads;
  float *ends = a.span_ends + kept * state, *into = a.span_backs + kept * state;
  Span span{j * a.span_chunks, j == last ? INT32_MAX : (j + 1) * a.span_chunks, nullptr, nullptr, moved};
  // what is walked as it is in the first launch, the other end, is not in the second
  if (second ? j == (adjoint ? last : 0) : j == (adjoint ? 0 : last) && last > 0) return;
  if constexpr (BACK) {
    if (adjoint) {
      if (j == last) span.from = state_of(a.ds_last, a, seq_head);
      else if (second) span.from = into;
      if (j == 0) span.to = state_of(a.ds0, a, seq_head);
      else if (!second) span.to = into - before;
      if (second || j == last) walk<IO, KD, NW, kBack>(a, sh.back, at.seq, head, vb0, span);
      else walk<IO, KD, NW, kBackSpan>(a, sh.back_part, at.seq, head, vb0, span);
      return;
    }
  }
  if (moved && j == 0) return;
  if (moved) {
    span.to = a.span_moves + kept * move;
  } else {
    if (j == 0) span.from = state_of(a.s0, a, seq_head);
    else if (second) span.from = ends - before;
    if (j == last) span.to = BACK ? nullptr : state_of(a.s_last, a, seq_head);
    else if (!second) span.to = ends;
  }
  if (second || j == 0) walk<IO, KD, NW, kWhole>(a, sh.whole, at.seq, head, vb0, span);
  else walk<IO, KD, NW, kPart>(a, sh.part, at.seq, head, vb0, span);
}

template <typename IO, int KD, int NW, bool BACK>
hipError_t launch_spans(const DeltaArgs& a, hipStream_t stream) {
  const uint32_t vblocks = (uint32_t)((a.vd + 16 * NW - 1) / (16 * NW)),
                 kblocks = (uint32_t)((a.kd + 16 * NW - 1) / (16 * NW)),
                 units = (uint32_t)a.spans * (uint32_t)a.heads;
  auto launch = [&](int second) {
    const uint32_t each = vblocks * (BACK ? 2 : 1) + (second ? 0 : kblocks);
    hipLaunchKernelGGL((delta_spans_kernel<IO, KD, NW, BACK>), dim3(units * each), dim3(64 * NW), 0, stream, a,
                       vblocks, kblocks, second);
    return hipGetLastError();
  };
  hipError_t e = launch(0);
  if (e == hipSuccess) e = launch_delta_span_states(a, stream);
  if (e == hipSuccess) e = launch(1);
  return e;
}
template <typename IO, int KD, int NW> hipError_t launch_spans(const DeltaArgs& a, hipStream_t stream) {
  return a.back ? launch_spans<IO, KD, NW, true>(a, stream) : launch_spans<IO, KD, NW, false>(a, stream);
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
    if constexpr (NW < 8) {  // (see waves_of)
      if (a.back)
        hipLaunchKernelGGL((delta_backward_kernel<IO, KD, NW>), grid, dim3(64 * NW), 0, stream, a, g, b);
    }
    if (!a.back)
      hipLaunchKernelGGL((delta_forward_kernel<IO, KD, NW>), grid, dim3(64 * NW), 0, stream, a, g, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Waves of a block, 16 value channels each.  Eight share one copy of the chunk's
// keys and triangles, but a CU has no room beside them; four leave room for a
// second block, and where there are few of either they spread over more CUs.  160
// heads of 128 over 4096 tokens 550 us in blocks of 8, 586 of 4; 32 heads over
// 65536 tokens 6.0 and 4.6 ms; the backward's two walks of the first 1.25 and 1.07
// ms.
inline int waves_of(const DeltaArgs& a) {
  if (a.vd <= 32) return 2;
  return !a.back && a.vd > 64 && a.nseq * a.heads * ((a.vd + 127) / 128) > 128 ? 8 : 4;
}

template <typename IO, int KD> hipError_t launch_kd(const DeltaArgs& a, hipStream_t stream) {
  if (a.span_chunks > 0)
    return a.vd <= 32 ? launch_spans<IO, KD, 2>(a, stream) : launch_spans<IO, KD, 4>(a, stream);
  switch (waves_of(a)) {
    case 2: return launch_nw<IO, KD, 2>(a, stream);
    case 4: return launch_nw<IO, KD, 4>(a, stream);
    default: return launch_nw<IO, KD, 8>(a, stream);
  }
}
template <typename IO> hipError_t launch_walk(const DeltaArgs& a, hipStream_t stream) {
  return a.kd <= 64 ? launch_kd<IO, 64>(a, stream) : launch_kd<IO, 128>(a, stream);
}

}  // namespace
}  // namespace ssm
