// ssm_linattn_mm.hip -- linear attention with one decay per head on the bf16
// matrix cores (gfx950, wave64): S_t = a S_{t-1} + v_t k_t^T, o_t = S_t q_t
// over whole sequences, in chunks of 64 tokens.
//
// Inside a chunk that the state S [vd, kd] enters, token t (0..63) reads
//   o_t = a^(t+1) S q_t + sum over s <= t of a^(t-s) (q_t . k_s) v_s
// and the chunk leaves  a^n S + sum over s of a^(n-1-s) v_s k_s^T:  four
// matrix products over the chunk instead of 64 rank-one updates.  A block of
// waves walks one unit (a sequence or a segment of one) of one head; each wave
// owns 16 value channels with the whole key dimension of their state in fp32
// accumulators, so the state never leaves the registers between chunks:
// its accumulator tile (rows: keys) is at the same time, rounded to bf16 parts,
// the operand of S q.  Only the chunk's weighted 64 x 64 products P, which
// every wave needs, go through LDS, beside the tiles of q, k, v.
//
// Bound by latency: of a chunk's 9,750 cycles for a block of 8 waves alone on
// its CU (heads of 128 x 128) the matrix cores are busy 3,100, the vector units
// 4,000 and LDS 3,700, one after the other between three barriers; a second
// block on the CU brings it to 6,250 a chunk.  Hence the layout: LDS for two
// blocks of 8 waves (64 KB each), 128 registers a wave, no spills, and loads of
// the next chunk that no barrier waits for.  Measured (copy rate 4.9 TB/s; boxes
// differ by 7%): 4 x 4096 tokens, 40 heads over 8, of 128: 223 us, 193 TFLOP/s
// and 1.8 TB/s of needed traffic; 16384 packed tokens, 80 heads of 128 x 64,
// with states: 267 us, 4.2 TB/s; 65536 tokens of 32 heads: 798 us, 4.0 TB/s with
// the state-only pass' second read of k and v; backward of the first: 663 us, of
// which 141 are the sums over shared heads; with the decay's gradient 1180.
// Chunks of 64: a token's share of the pair product grows with the chunk, that of
// the state's conversions and of the barriers falls with it.  Two value tiles a
// wave in blocks of 4 waves halve the LDS reads of q, k and P but take as long with
// two blocks on a CU (265 against 265 us) and longer with one (314 against 281).
//
// Precision: q, k, v are bf16 and enter as they are.  S and P enter o, which is
// rounded to bf16, as two bf16 parts (16 bits), and the decay's gradient, which
// is fp32, as three.  Weighted v enters every state as three (24 bits), also
// those of dq and dk, which no output holds: they are carried over the whole
// sequence.  Two would save a sixth of their matrix work (the backward above 5%)
// and move one in 2700 bf16 gradients to its neighbour.
#include <algorithm>

#include "ssm_linattn_walk.h"
#include "ssm_mfma.h"

namespace ssm {
namespace {

constexpr int C = kLinChunk;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// Transposing LDS read: in each group of 16 lanes, lane i gives the address of
// 4 consecutive elements (row i / 4, columns 4 (i % 4)..) and receives column
// i of the 4 rows.
__device__ __forceinline__ u32x2_t lds_tr(const uint8_t* p, uint32_t off) {
  return __builtin_bit_cast(u32x2_t,
                            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + off)));
}

__device__ __forceinline__ float part_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float part_lo(uint32_t w) { return __uint_as_float(w << 16); }

// One bf16 part of 8 values and what it leaves of them, by the two-term dot
// product of bf16 pairs (x - w * 1, exact): one instruction for unpacking and
// subtracting.
__device__ __forceinline__ u32x4_t take_parts(float* x) {
  bf16x2_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = bf16x2_t{(__bf16)x[2 * i], (__bf16)x[2 * i + 1]};
  // The pairs (-1, 0) and (0, -1) are kept from the compiler: it writes the
  // first as the inline constant -1.0, which the instruction reads as the second.
  uint32_t lo = 0x0000bf80u, hi = 0xbf800000u;
  asm("" : "+s"(lo), "+s"(hi));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = __builtin_amdgcn_fdot2_f32_bf16(w[i / 2], __builtin_bit_cast(bf16x2_t, i & 1 ? hi : lo),
                                           x[i], false);
  return u32x4_t{__builtin_bit_cast(uint32_t, w[0]), __builtin_bit_cast(uint32_t, w[1]),
                 __builtin_bit_cast(uint32_t, w[2]), __builtin_bit_cast(uint32_t, w[3])};
}
__device__ __forceinline__ u32x4_t last_parts(const float* x) {
  return u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                 pack_bf16(x[6], x[7])};
}

// Whether any of a tile's pieces holds an infinity or a NaN.
template <int N> __device__ __forceinline__ bool any_odd(const u32x4_t (&r)[N]) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  u16x2_t m = {0, 0};
#pragma unroll
  for (int p = 0; p < N; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, r[p][i] & 0x7fff7fffu));
  return m[0] >= 0x7f80 || m[1] >= 0x7f80;
}

// Byte address of element (row, col) of a [rows, W] bf16 tile in LDS.  Rows
// are not padded; instead the 32-byte pieces of every 256 bytes are exchanged
// by the row, which leaves both the row reads (16 bytes of 16 rows a lane
// group) and the transposing reads (32 bytes of 4 rows a lane group) without
// bank conflicts.
template <int W> __device__ __forceinline__ uint32_t at(int row, int col) {
  const uint32_t b = (uint32_t)(row * W + col) * 2;
  return b ^ (uint32_t)(((W >= 128 ? row : row >> 1) & 7) << 5);
}
typedef uint8_t lds_byte;
__device__ __forceinline__ u32x4_t ld128(const lds_byte* p, uint32_t off) {
  return *reinterpret_cast<const u32x4_t*>(p + off);
}
__device__ __forceinline__ u32x2_t ld64(const lds_byte* p, uint32_t off) {
  return *reinterpret_cast<const u32x2_t*>(p + off);
}

// Units of packed sequences: their number, pairs (sequence, segment), then
// every sequence's first unit.  A sequence's units are consecutive, and the
// longest sequences come first, so that the blocks that take longest start
// first (a sequence without tokens has one unit).  One block sorts by the
// number of chunks: counted from the most down, then placed, equal ones in
// their order (the parts of the decay's gradient are added in that of the units).
// Sums are 64-bit: cu_seqlens that run up and down make sequences that overlap,
// and their units may be more than 2^31 (those past the table's end are left out).
constexpr int kBuckets = 1024;
__global__ __launch_bounds__(kBuckets) void unit_table_kernel(LinArgs a) {
  typedef unsigned long long Count;
  __shared__ Count start[kBuckets];
  __shared__ Count run[kBuckets / 64];
  __shared__ int2 mine[kBuckets];  // bucket and units of a round's sequences
  __shared__ int held[2];          // first token of any sequence, end of the last
  const int i = threadIdx.x, most = (int)a.units;
  auto units_of = [&](int seq, int& bucket, int& first, int& len) {
    sequence_of(a, seq, first, len);
    const int chunks = (int)(((int64_t)len + C - 1) / C);
    bucket = kBuckets - 1 - min(chunks, kBuckets - 1);
    return segments_of(a, len);
  };
  start[i] = 0;
  if (i == 0) held[0] = (int)a.tokens, held[1] = 0;
  __syncthreads();
  int lo = (int)a.tokens, hi = 0;
  for (int s = i; s < a.nseq; s += kBuckets) {
    int b, first, len;
    const int n = units_of(s, b, first, len);
    atomicAdd(&start[b], (Count)n);
    if (len > 0) lo = min(lo, first), hi = max(hi, first + len);
  }
  for (int d = 1; d < 64; d <<= 1) {
    lo = min(lo, __shfl_xor(lo, d));
    hi = max(hi, __shfl_xor(hi, d));
  }
  if ((i & 63) == 0 && lo < hi) {
    atomicMin(&held[0], lo);
    atomicMax(&held[1], hi);
  }
  __syncthreads();
  // sums over the buckets up to each: within waves, then of the waves before
  const Count count = start[i];
  Count upto = count;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const Count v = __shfl_up(upto, d);
    if ((i & 63) >= d) upto += v;
  }
  if ((i & 63) == 63) run[i >> 6] = upto;
  __syncthreads();
  Count total = 0;
#pragma unroll
  for (int w = 0; w < kBuckets / 64; ++w) {
    if (w < (i >> 6)) upto += run[w];
    total += run[w];
  }
  start[i] = upto - count;
  __syncthreads();
  for (int s0 = 0; s0 < a.nseq; s0 += kBuckets) {
    const int s = s0 + i;
    int b = -1, n = 0, first, len;
    if (s < a.nseq) n = units_of(s, b, first, len);
    mine[i] = int2{b, n};
    __syncthreads();
    if (n > 0) {
      Count at = start[b];
      for (int j = 0; j < i; ++j) at += (Count)(mine[j].x == b ? mine[j].y : 0);
      const int to = (int)min(at, (Count)most);
      a.unit_table[1 + 2 * (int64_t)most + s] = to;
      for (int k = 0; k < n && to + k < most; ++k) {
        a.unit_table[1 + 2 * (int64_t)(to + k)] = s;
        a.unit_table[2 + 2 * (int64_t)(to + k)] = k;
      }
    }
    __syncthreads();
    if (n > 0) atomicAdd(&start[b], (Count)n);
    __syncthreads();
  }
  if (i == 0) a.unit_table[0] = (int)min(total, (Count)most);
  if (i < 2) a.unit_table[lin_table_ints(most, a.nseq) - 2 + i] = held[i];
}

// A [64, W] bf16 tile on its way into LDS: 16-byte pieces in registers.
template <int W, int THREADS> struct Tile {
  static constexpr int kPerRow = W / 8;
  static constexpr int kRows = THREADS / kPerRow;  // rows per pass
  static constexpr int kPasses = C / kRows;
  u32x4_t r[kPasses];

  // Byte offset of the lane's first piece: row threadIdx.x / kPerRow, or out of
  // range past the operand's channels, where buffer loads read zero.
  __device__ __forceinline__ static uint32_t start(int64_t stride, int col0, int dim, uint32_t tid) {
    const int c = (tid % kPerRow) * 8 + col0;
    return c < dim ? (tid / kPerRow) * (uint32_t)stride * 2 + (uint32_t)c * 2 : 0x7f000000u;
  }
  // Rows 0..n-1 from `base`, in memory order; rows past n read zero (a chunk's
  // 64 rows span less than 2^30 bytes, so no offset wraps).
  __device__ __forceinline__ void load(const bf16* base, int64_t stride, int n, int dim,
                                       uint32_t start) {
    const uint32_t sb = (uint32_t)stride * 2;
    const __amdgpu_buffer_rsrc_t rsrc =
        make_rsrc(base, n > 0 ? (uint32_t)(n - 1) * sb + (uint32_t)dim * 2 : 0u);
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      r[p] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rsrc, start + p * kRows * sb, 0, 0));
  }
  __device__ __forceinline__ void store(lds_byte* lds, uint32_t tid) const {
    const int c = (tid % kPerRow) * 8, row = tid / kPerRow;
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      *reinterpret_cast<u32x4_t*>(lds + at<W>(row, c) + p * kRows * W * 2) = r[p];
  }
  // Channels of each 32 reordered so that 16 bytes at 8 g hold channels
  // 4g..4g+3 and 16+4g..16+4g+3: the rows that lane group g has of two stacked
  // accumulator tiles.
  __device__ __forceinline__ void store_paired(lds_byte* lds, uint32_t tid) const {
    const int c8 = tid % kPerRow, row = tid / kPerRow;
    const uint32_t a = at<W>(row, (c8 / 4) * 32 + (c8 & 1) * 16 + ((c8 >> 1) & 1) * 4);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      lds_byte* d = lds + a + p * kRows * W * 2;
      *reinterpret_cast<u32x2_t*>(d) = u32x2_t{r[p].x, r[p].y};
      *reinterpret_cast<u32x2_t*>(d + 16) = u32x2_t{r[p].z, r[p].w};
    }
  }
};

// The ten 16 x 16 tiles (tt, st) of P with a pair in walk order (st <= tt;
// going back st >= tt): tiles of wave w of NW.
template <int NW> __device__ __forceinline__ int pair_tiles(int w) {
  return NW == 8 ? (w < 2 ? 2 : 1) : (w < 2 ? 3 : 2);
}
template <int NW, bool REV> __device__ __forceinline__ void pair_tile(int w, int i, int& tt, int& st) {
  if (NW == 8) {  // (0, 0), (1, 0), (1, 1), (2, 0..2), (3, 0), (3, 1); (3, 2), (3, 3)
    const int n = w + 8 * i;
    tt = n == 0 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3;
    st = n - (tt == 0 ? 0 : tt == 1 ? 1 : tt == 2 ? 3 : 6);
  } else if (w < 2) {  // (3, 0..2), (2, 0..2)
    tt = 3 - w;
    st = i;
  } else if (w == 2) {  // (3, 3), (1, 0)
    tt = i ? 1 : 3;
    st = i ? 0 : 3;
  } else {  // (0, 0), (1, 1)
    tt = st = i;
  }
  if (REV) {
    tt = 3 - tt;
    st = 3 - st;
  }
}

template <int KD, int VB, bool MAIN, bool TAN> struct alignas(256) Shared {
  lds_byte k[C * KD * 2];
  lds_byte v[C * VB * 2];
  lds_byte q[MAIN ? C * KD * 2 : 16];
  lds_byte p[TAN ? 3 : 2][MAIN ? C * C * 2 : 16];  // parts, [t][s] with s as in store_paired
  // by row of the chunk: weights of v on its way into the state (a^(n-1-s);
  // going back a^(s+1)) and of S q (a^(t+1); going back a^(n-1-t))
  float w[C];
  float rw[MAIN ? C : 1];
  double part[TAN ? 4 * VB : 1];         // sums of the block's threads
  float pw[MAIN ? C + 16 : 1];           // pw[63 - d]: weight of a pair d tokens apart, d > -16
  int odd[2];                            // whether v holds an infinity or NaN, by chunk parity
};

// Waves a SIMD has to hold: as many as the LDS leaves room for; the walk that
// carries the state's derivative keeps twice the state.
constexpr int waves_per_simd(int kd, int nw, bool state, bool tan) {
  return kd > 128 || tan ? nw / 4 : nw == 8 || state ? 4 : kd > 64 ? 2 : 3;
}

// One block's walk over the unit u of one head, value channels vb0 on.  MAIN:
// with outputs, else the state alone.  TAN: for the derivative by the log
// decay g the state's derivative T = dS/dg is carried too,
//   T <- a^n (T + n S) + sum over s of (n-1-s) a^(n-1-s) v_s k_s^T,
// and what is summed is dy_t . do_t/dg with
//   do_t/dg = a^(t+1) ((t+1) S + T) q_t + sum of (t-s) a^(t-s) (q_t . k_s) v_s.
template <int KD, int NW, bool MAIN, bool REV, bool TAN>
__device__ __forceinline__ void walk(const LinArgs& a, Shared<KD, 16 * NW, MAIN, TAN>& sh,
                                     const Unit& x, uint32_t u, int head, int vb0,
                                     uint32_t part_at) {
  constexpr int VB = 16 * NW, RT = KD / 16, KS = KD / 32;
  constexpr int PP = TAN ? 3 : 2;  // parts of P, S and T in the outputs' products
  constexpr int PARTS = 3;         // of weighted v in the states'
  const bool last_unit = x.p0 + x.n >= x.len;
  if (!MAIN && last_unit) return;  // its end state is the walk's

  const int64_t uh = (int64_t)u * a.heads + head;
  const int w = wave_id(), lane = threadIdx.x & 63;
  int r16 = lane & 15, g = lane >> 4;
  uint32_t tid = threadIdx.x;
  const float g2 = log2_decay(a.log_decay[head]);
  const int dv0 = w * 16;  // the wave's value channels in the block's

  // S[rt]: keys 16 rt + 4 g + i of the wave's channel r16.  Outside the state's
  // channels it is zero.
  const int dvs = vb0 + dv0 + r16;
  f32x4_t S[RT], T[TAN ? RT : 1];
  const int64_t state = (int64_t)a.vd * a.kd, seq_state = ((int64_t)x.seq * a.heads + head) * state;
  const uint32_t state_bytes = (uint32_t)state * 4;
  {
    // what enters the segment; folded, the first segment's end
    const bool inner = MAIN && x.p0 > 0;
    const int64_t slot = (uh - (a.fold ? (int64_t)x.seg * a.heads : 0)) * state;
    const float* from = inner ? a.ws_state + slot : a.s0 + seq_state;
    const bool given = x.seg == 0 && a.s0;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(from, inner || given ? state_bytes : 0u);
    const bool swap = a.s0_swap && !inner;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int dk = 16 * rt + 4 * g;
      const bool on = dvs < a.vd && dk < a.kd;
      if constexpr (TAN) {
        const __amdgpu_buffer_rsrc_t rt_ =
            make_rsrc(a.ws_tangent + slot, inner ? state_bytes : 0u);
        T[rt] = __builtin_bit_cast(
            f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                         rt_, on ? (uint32_t)(dvs * a.kd + dk) * 4 : 0x7f000000u, 0, 0));
      }
      if (!swap) {
        S[rt] = __builtin_bit_cast(
            f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                         rs, on ? (uint32_t)(dvs * a.kd + dk) * 4 : 0x7f000000u, 0, 0));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          S[rt][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
              rs, on ? (uint32_t)((dk + i) * a.vd + dvs) * 4 : 0x7f000000u, 0, 0));
      }
    }
  }

  if (!MAIN && x.seg == 0) {  // what the segment leaves of the given state
    const float as = power(g2, x.n);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      S[rt] *= as;
      if constexpr (TAN) T[rt] = (float)x.n * S[rt];
    }
  }
  if (MAIN && x.seg > 1 && a.fold) {  // join the segments between
    const Decays all = wave_decays(a.log_decay[head], x.seg_len);
    for (int j = x.seg - 1; j > 0; --j) {
      const float as = decay_of(all, x.seg - 1 - j);
      const int64_t slot = (uh - (int64_t)j * a.heads) * state;
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.ws_state + slot, state_bytes);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int dk = 16 * rt + 4 * g;
        const uint32_t from =
            dvs < a.vd && dk < a.kd ? (uint32_t)(dvs * a.kd + dk) * 4 : 0x7f000000u;
        if constexpr (TAN)
          T[rt] = as * (T[rt] + (float)x.seg_len * S[rt]) +
                  __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                  make_rsrc(a.ws_tangent + slot, state_bytes),
                                                  from, 0, 0));
        const f32x4_t own =
            __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, from, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) S[rt][i] = __builtin_fmaf(as, S[rt][i], own[i]);
      }
    }
  }

  const bf16* qp = static_cast<const bf16*>(a.q.p) + (int64_t)(head / a.q.hdiv) * a.kd;
  const bf16* kp = static_cast<const bf16*>(a.k.p) + (int64_t)(head / a.k.hdiv) * a.kd;
  const bf16* vp = static_cast<const bf16*>(a.v.p) + (int64_t)(head / a.v.hdiv) * a.vd;
  uint32_t q_at = Tile<KD, 64 * NW>::start(a.q.stride, 0, a.kd, tid);
  uint32_t k_at = Tile<KD, 64 * NW>::start(a.k.stride, 0, a.kd, tid);
  uint32_t v_at = Tile<VB, 64 * NW>::start(a.v.stride, vb0, a.vd, tid);
  const int end = x.p0 + x.n;
  // First token in memory of the chunk of n tokens at walk position c0.  The
  // state alone is gathered from the segment's last chunk to its first (whole
  // chunks), each weighted by its distance from the end, so that the main pass
  // finds in the caches what was read last: 65536 tokens of 32 heads of 128
  // 813 -> 801 us.
  auto token0 = [&](int c0, int n) {
    const int c = MAIN ? c0 : end - C - (c0 - x.p0);
    return x.first + (REV ? x.len - c - n : c);
  };

  Tile<KD, 64 * NW> tq, tk;
  Tile<VB, 64 * NW> tv;
  // the tiles of the chunk at c0 (none past the unit's end: zeros, unread)
  auto load_q = [&](int c0, int n) {
    if constexpr (MAIN)
      tq.load(qp + (uint64_t)(uint32_t)token0(c0, n) * (uint32_t)a.q.stride, a.q.stride, n, a.kd,
              q_at);
  };
  auto load_k = [&](int c0, int n) {
    tk.load(kp + (uint64_t)(uint32_t)token0(c0, n) * (uint32_t)a.k.stride, a.k.stride, n, a.kd,
            k_at);
  };
  auto load_v = [&](int c0, int n) {
    tv.load(vp + (uint64_t)(uint32_t)token0(c0, n) * (uint32_t)a.v.stride, a.v.stride, n, a.vd,
            v_at);
  };
  auto size = [&](int c0) { return c0 >= end ? 0 : end - c0 < C ? end - c0 : C; };

  if constexpr (MAIN) {
    // tiles that share a product's 32 rows with the diagonal tile but have no
    // pair in walk order: zero, never written again
    if (threadIdx.x < 128) {
      const int e = threadIdx.x, row = 32 * (e >> 6) + (REV ? 16 : 0) + (e & 15);
      const int col = 32 * (e >> 6) + 8 * ((e >> 4) & 3) + (REV ? 0 : 4);
#pragma unroll
      for (int i = 0; i < PP; ++i)
        *reinterpret_cast<u32x2_t*>(sh.p[i] + at<C>(row, col)) = u32x2_t{0, 0};
    }
    if (threadIdx.x < 2) sh.odd[threadIdx.x] = 0;
    if (threadIdx.x < C + 16) {
      const int d = 63 - (int)threadIdx.x;
      sh.pw[threadIdx.x] =
          power(g2, d > 0 ? d : 0) * (TAN ? a.pair_scale * (float)d : a.pair_scale);
    }
  }

  // A chunk's o stands in v's tile when the chunk is done, each wave's in the
  // channels that it alone read, and leaves from there in whole rows (stored
  // from the accumulators, 32 bytes of 16 rows at a time, a chunk's 16 KB keep
  // the memory pipe for 2370 cycles of a CU, in rows of 256 bytes for 850).  A
  // thread takes exactly the pieces that it will fill with the next tile.
  const bool staged = MAIN && !TAN && !a.o_f32;
  auto leave = [&](int c0, int n, const Tile<VB, 64 * NW>* next) {
    typedef Tile<VB, 64 * NW> V;
    u32x4_t o[V::kPasses];
    const uint32_t slot = at<VB>(tid / V::kPerRow, (tid % V::kPerRow) * 8);
#pragma unroll
    for (int p = 0; p < V::kPasses; ++p) o[p] = ld128(sh.v, slot + p * V::kRows * VB * 2);
    if (next) next->store(sh.v, tid);
    const uint32_t row = (uint32_t)a.heads * a.vd * 2;  // rows past n are dropped
    const __amdgpu_buffer_rsrc_t ro =
        make_rsrc(static_cast<bf16*>(a.o) + ((int64_t)token0(c0, n) * a.heads + head) * a.vd,
                  (uint32_t)(n - 1) * row + (uint32_t)a.vd * 2);
    const uint32_t to = V::start((int64_t)a.heads * a.vd, vb0, a.vd, tid);
#pragma unroll
    for (int p = 0; p < V::kPasses; ++p)
      __builtin_amdgcn_raw_buffer_store_b128(o[p], ro, to + p * V::kRows * row, 0, 0);
  };

  // of whole chunks, where there are several
  const float g_chunk = scalar(power(g2, C));
  Decays chunk_decays{g_chunk, g_chunk, 0.0f};
  if (MAIN && !TAN && x.n > C) chunk_decays = wave_decays(a.log_decay[head], C);

  double dg = 0.0;  // the lane's part of the sum (TAN)
  {
    const int n = size(x.p0);
    load_q(x.p0, n);
    load_k(x.p0, n);
    load_v(x.p0, n);
  }
  if constexpr (MAIN) lds_barrier();  // odd is cleared
  for (int c0 = x.p0; c0 < end; c0 += C) {
    const int n = size(c0);
    // Addresses are derived from these anew in every chunk: kept over the loop
    // they would push the state out of the registers.
    asm volatile("" : "+v"(r16), "+v"(g), "+v"(tid), "+v"(q_at), "+v"(k_at), "+v"(v_at));
    if (c0 > x.p0) lds_barrier();  // the previous chunk's tiles are read, its o is whole
    if constexpr (MAIN) tq.store_paired(sh.q, tid);
    tk.store(sh.k, tid);
    if (staged && c0 > x.p0) {
      leave(c0 - C, C, &tv);
    } else {
      tv.store(sh.v, tid);
    }
    const int parity = ((c0 - x.p0) / C) & 1;
    if constexpr (MAIN) {
      if (any_odd(tv.r)) sh.odd[parity] = 1;
    }
    if (c0 == x.p0 || n < C) {
      if (threadIdx.x < C) {
        const int i = threadIdx.x, left = i < n ? n - 1 - i : 0;
        // rows past n are no tokens; a growing decay's power may be infinite there
        sh.w[i] = i < n ? power(g2, REV ? i + 1 : left) * a.write_scale : 0.0f;
        if constexpr (MAIN) sh.rw[i] = i < n ? power(g2, REV ? left : i + 1) * a.read_scale : 0.0f;
      }
    }
    lds_barrier();
    // The next chunk's tiles are asked for between this one's products: all at
    // once they would hold the waves up at the memory pipe.
    const int c1 = c0 + C < end ? c0 + C : c0, n1 = size(c0 + C);
    if constexpr (!MAIN) {
      load_k(c1, n1);
      load_v(c1, n1);
    }

    f32x4_t acc[4];  // [tt]: token 16 tt + r16, channels 4 g + i of the wave's
    float gn = g2;
    asm volatile("" : "+v"(gn));  // nor is the decay of a whole chunk
    // of the whole chunk; going for the state alone, of what follows the chunk
    const float an = MAIN && !TAN && n == C ? decay_of(chunk_decays, (c0 - x.p0) / C)
                                            : power(gn, MAIN ? n : c0 - x.p0);
    // The decay's gradient takes in the decays of many chunks, each off by the
    // same rounding of a^n; so that goes by with what it leaves, and the sum is
    // carried in 64 bits over the chunks: 5.2e-7 of the gradient, 6.3e-7 without,
    // 7.2e-7 in plain fp32 (rms over 12 inputs, 8 x 2048 tokens of 24 heads of 64).
    float an_rest = 0.0f;
    if constexpr (MAIN && TAN) {
      const double all = exp2((double)a.log_decay[head] * 1.4426950408889634 * n);
      an_rest = an <= 3e38f ? (float)(all - (double)an) : 0.0f;  // (more is infinite anyway)
    }
    const uint32_t qa = at<KD>(r16, 8 * g);
    if constexpr (MAIN) {
      // P: rows s of k against columns t of q, so that a lane holds 4
      // consecutive s of one t
      const uint32_t ka = at<KD>(r16, 4 * g);
      constexpr int NP = NW == 8 ? 2 : 3;
      const int np = pair_tiles<NW>(w);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (i < np) {
          int tt, st;
          pair_tile<NW, REV>(w, i, tt, st);
          f32x4_t m{0, 0, 0, 0};
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            m = mfma_k32(cat(ld64(sh.k, (ka ^ (64 * ks)) + 16 * st * KD * 2),
                             ld64(sh.k, (ka ^ (64 * ks + 32)) + 16 * st * KD * 2)),
                         ld128(sh.q, (qa ^ (64 * ks)) + 16 * tt * KD * 2), m);
          const int ts = 16 * (tt - st) + r16 - 4 * g;  // t - s of the first s
          // going back, rows past n come before t: no tokens, but the weight of
          // such a pair may be infinite (a decay that grows)
          const int rows = REV ? n - 16 * st - 4 * g : C;
          float v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = REV ? j - ts : ts - j;
            v[j] = m[j] * sh.pw[63 - d];
            v[j] = d >= 0 && j < rows ? v[j] : 0.0f;  // a select: the pair may be infinite or NaN
          }
          const uint32_t to = at<C>(16 * tt + r16, 32 * (st >> 1) + 8 * g + 4 * (st & 1));
#pragma unroll
          for (int part = 0; part < PP; ++part) {
            const u32x2_t b = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            *reinterpret_cast<u32x2_t*>(sh.p[part] + to) = b;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] -= j & 1 ? part_hi(b[j / 2]) : part_lo(b[j / 2]);
          }
        }
      }
      load_q(c1, n1);
      // acc = S q, weighted (S and T are scaled on the way)
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) acc[tt] = f32x4_t{0, 0, 0, 0};
      f32x4_t tq_[TAN ? 4 : 1];  // T q
      if constexpr (TAN) {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) tq_[tt] = f32x4_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        f32x4_t &s0 = S[2 * ks], &s1 = S[2 * ks + 1];
        if (ks == KS / 2) load_k(c1, n1);
        u32x4_t sp[PP], tp[TAN ? PP : 1];
        auto parts_of = [](f32x4_t x, f32x4_t y, u32x4_t* to) {
          float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
          for (int i = 0; i < PP; ++i) to[i] = i + 1 < PP ? take_parts(z) : last_parts(z);
        };
        parts_of(s0, s1, sp);
        if constexpr (TAN) {
          f32x4_t &t0 = T[2 * ks], &t1 = T[2 * ks + 1];
          parts_of(t0, t1, tp);
          t0 += (float)n * s0;
          t1 += (float)n * s1;
          t0 = an * t0 + an_rest * t0;
          t1 = an * t1 + an_rest * t1;
          s0 = an * s0 + an_rest * s0;
          s1 = an * s1 + an_rest * s1;
        }
        u32x4_t b[4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) b[tt] = ld128(sh.q, (qa ^ (64 * ks)) + 16 * tt * KD * 2);
#pragma unroll
        for (int i = 0; i < PP; ++i)
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) {
            acc[tt] = mfma_k32(sp[i], b[tt], acc[tt]);
            if constexpr (TAN) tq_[tt] = mfma_k32(tp[i], b[tt], tq_[tt]);
          }
      }
      if constexpr (TAN) {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) acc[tt] = (float)(16 * tt + r16 + 1) * acc[tt] + tq_[tt];
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) acc[tt] *= sh.rw[16 * tt + r16];
    }

    // v of the wave's channels, tokens 32 ks + {4g.., 16 + 4g..} in the slots
    u32x4_t vo[2];
    const uint32_t va = at<VB>(4 * g + (r16 >> 2), dv0 + 4 * (r16 & 3));
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      vo[ks] = cat(lds_tr(sh.v, va + 32 * ks * VB * 2), lds_tr(sh.v, va + (32 * ks + 16) * VB * 2));
    int any = 0;
    if constexpr (MAIN) {
      any = sh.odd[parity];
      lds_barrier();  // P is whole
      load_v(c1, n1);
      if (threadIdx.x == 0) sh.odd[parity ^ 1] = 0;
    }

    int first = REV ? -1 : C;  // of channel r16, the first token (in walk order) with an odd value
    bool odd = false;
    if constexpr (MAIN) {
      // A later token's infinity or NaN must not reach an earlier one through
      // its zero weight: such values enter the products as zeros, and the
      // tokens that read them, and the state, become NaN at the end.
      odd = __builtin_amdgcn_readfirstlane(any) != 0;
      if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t e = vo[ks][j / 2], mask = j & 1 ? 0xffff0000u : 0xffffu;
            if ((e & mask & 0x7f807f80u) == (mask & 0x7f807f80u)) {
              const int s = 32 * ks + 16 * (j / 4) + 4 * g + (j & 3);
              first = REV ? max(first, s) : min(first, s);
              vo[ks][j / 2] = e & ~mask;
            }
          }
#pragma unroll
        for (int m = 16; m < 64; m <<= 1) {
          const int other = __shfl_xor(first, m);
          first = REV ? max(first, other) : min(first, other);
        }
      }
      const uint32_t pa = at<C>(r16, 8 * g);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int part = 0; part < PP; ++part)
#pragma unroll
          for (int tt = REV ? 0 : 2 * ks; tt < (REV ? 2 * ks + 2 : 4); ++tt)
            acc[tt] = mfma_k32(vo[ks], ld128(sh.p[part], (pa ^ (64 * ks)) + 16 * tt * C * 2),
                               acc[tt]);
      if (__builtin_expect(odd, 0)) {
        const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int f = __shfl(first, 4 * g + i);
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
            if (REV ? 16 * tt + r16 <= f : 16 * tt + r16 >= f) acc[tt][i] = nan;
        }
      }
      const int dv = vb0 + dv0 + 4 * g;
      if constexpr (TAN) {
        // dy of the same tokens and channels, zero where there is none
        const uint32_t row = (uint32_t)a.dy.stride * 2;
        const __amdgpu_buffer_rsrc_t ry = make_rsrc(
            static_cast<const bf16*>(a.dy.p) +
                (uint64_t)(uint32_t)token0(c0, n) * (uint32_t)a.dy.stride + (int64_t)head * a.vd,
            (uint32_t)(n - 1) * row + (uint32_t)a.vd * 2);
        float here = 0.0f;
        const uint32_t ya = dv < a.vd ? r16 * row + (uint32_t)dv * 2 : 0x7f000000u;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const u32x2_t y = __builtin_bit_cast(
              u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(ry, ya + 16 * tt * row, 0, 0));
          if (16 * tt + r16 < n && dv < a.vd) {
            here = __builtin_fmaf(acc[tt][0], part_lo(y.x), here);
            here = __builtin_fmaf(acc[tt][1], part_hi(y.x), here);
            here = __builtin_fmaf(acc[tt][2], part_lo(y.y), here);
            here = __builtin_fmaf(acc[tt][3], part_hi(y.y), here);
          }
        }
        dg += (double)here;
      } else {
        // a lane holds 4 consecutive channels of 4 tokens
        if (staged) {
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
            *reinterpret_cast<u32x2_t*>(sh.v + at<VB>(16 * tt + r16, dv0 + 4 * g)) =
                to_bf16x4(acc[tt]);
        } else {  // fp32, 64 bytes of 16 rows at a time
          const uint32_t row = (uint32_t)a.heads * a.vd * 4;
          const __amdgpu_buffer_rsrc_t ro =
              make_rsrc(static_cast<float*>(a.o) + ((int64_t)token0(c0, n) * a.heads + head) * a.vd,
                        (uint32_t)(n - 1) * row + (uint32_t)a.vd * 4);
          const uint32_t oa = dv < a.vd ? r16 * row + (uint32_t)dv * 4 : 0x7f000000u;
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[tt]), ro,
                                                   oa + 16 * tt * row, 0, 0);
        }
      }
    }

    // S <- a^n S + k^T (w v); S + a^.. k^T (w v).  The parts are added up first,
    // the last one first: into a state of many chunks the small ones would be
    // lost, and where all weights are near 1 they have one sign (65536 tokens at
    // a decay of 3e-6: the state 5e-5 off on average; 1e-7 so).
    uint32_t kt = at<KD>(4 * g + (r16 >> 2), 4 * (r16 & 3));
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      asm volatile("" : "+v"(kt));  // its eight variants are not kept over both halves
      u32x4_t part[PARTS], tpart[TAN ? PARTS : 1];
      f32x4_t w0 = *reinterpret_cast<const f32x4_t*>(sh.w + 32 * ks + 4 * g);
      f32x4_t w1 = *reinterpret_cast<const f32x4_t*>(sh.w + 32 * ks + 16 + 4 * g);
      if constexpr (!MAIN) w0 *= an, w1 *= an;
      float wv[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wv[2 * i] = part_lo(vo[ks][i]) * (i < 2 ? w0[2 * i] : w1[2 * i - 4]);
        wv[2 * i + 1] = part_hi(vo[ks][i]) * (i < 2 ? w0[2 * i + 1] : w1[2 * i - 3]);
      }
      if constexpr (TAN) {  // rows past n are zero
        const int far = MAIN ? n - 1 : c0 - x.p0 + C - 1;  // decays of the chunk's first token
        float tv_[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          tv_[j] = wv[j] * (float)(far - (32 * ks + 16 * (j / 4) + 4 * g + (j & 3)));
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
          tpart[p] = p + 1 < PARTS ? take_parts(tv_) : last_parts(tv_);
      }
#pragma unroll
      for (int p = 0; p < PARTS; ++p) part[p] = p + 1 < PARTS ? take_parts(wv) : last_parts(wv);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const u32x4_t ko = cat(lds_tr(sh.k, (kt ^ (32 * rt)) + 32 * ks * KD * 2),
                               lds_tr(sh.k, (kt ^ (32 * rt)) + (32 * ks + 16) * KD * 2));
        f32x4_t d{0, 0, 0, 0}, td{0, 0, 0, 0};
#pragma unroll
        for (int p = PARTS - 1; p >= 0; --p) {
          d = mfma_k32(ko, part[p], d);
          if constexpr (TAN) td = mfma_k32(ko, tpart[p], td);
        }
        if constexpr (TAN) T[rt] += td;
        if (MAIN && !TAN && ks == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) S[rt][j] = __builtin_fmaf(an, S[rt][j], d[j]);
        } else {
          S[rt] += d;
        }
      }
    }

    if (MAIN && __builtin_expect(odd, 0) && (REV ? first >= 0 : first < C)) {
      const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        S[rt] = f32x4_t{nan, nan, nan, nan};
        if constexpr (TAN) T[rt] = S[rt];
      }
    }
  }

  if (staged && x.n > 0) {
    lds_barrier();
    const int n = (x.n - 1) % C + 1;
    leave(end - n, n, nullptr);
  }
  if constexpr (MAIN && TAN) {
    if (a.ds_last && last_unit) {
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.ds_last + seq_state, state_bytes);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int dk = 16 * rt + 4 * g;
        const f32x4_t d = __builtin_bit_cast(
            f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                         rs, dvs < a.vd && dk < a.kd ? (uint32_t)(dvs * a.kd + dk) * 4
                                                     : 0x7f000000u, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) dg += (double)(T[rt][i] * d[i]);
      }
    }
    sh.part[threadIdx.x] = dg;
    __syncthreads();
    for (int m = 32 * NW; m > 0; m >>= 1) {
      if ((int)threadIdx.x < m) sh.part[threadIdx.x] += sh.part[threadIdx.x + m];
      __syncthreads();
    }
    if (threadIdx.x == 0) a.dg_part[part_at] = (float)sh.part[0];
  }
  // the result, or a segment's end for those after it
  const bool between = !last_unit && (!MAIN || (a.lead && x.seg == 0));
  if (!between && (TAN || !last_unit || !a.s_last)) return;
  const __amdgpu_buffer_rsrc_t rs =
      make_rsrc(between ? a.ws_state + uh * state : a.s_last + seq_state, state_bytes);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int dk = 16 * rt + 4 * g;
    const uint32_t to = dvs < a.vd && dk < a.kd ? (uint32_t)(dvs * a.kd + dk) * 4 : 0x7f000000u;
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, S[rt]), rs, to, 0, 0);
    if constexpr (TAN)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, T[rt]),
                                             make_rsrc(a.ws_tangent + uh * state, state_bytes), to,
                                             0, 0);
  }
}

// The unit and head of a block of n walks, and its first value channel.
struct Block {
  Unit x;
  uint32_t u;
  int head, vb0;
  uint32_t part_at;
  bool on;  // there is such a unit
};
template <int VB>
__device__ __forceinline__ Block block_of(const LinArgs& a, uint32_t r, uint32_t vblocks,
                                          uint32_t place0) {
  Block b;
  const uint32_t ph = r / vblocks, vb = r - ph * vblocks, place = ph / (uint32_t)a.heads;
  b.u = unit_at(a, place0 + place);
  b.head = (int)(ph - place * (uint32_t)a.heads);
  b.vb0 = (int)vb * VB;
  b.part_at = (b.u * vblocks + vb) * (uint32_t)a.heads + (uint32_t)b.head;
  b.on = unit_of(a, b.u, b.x);
  return b;
}

// LDS of a pass' blocks: of walks, of states, of either.
template <int KD, int NW, Pass PASS, bool TAN> union Storage {
  Shared<KD, 16 * NW, PASS != kState, TAN> main;
  Shared<KD, 16 * NW, false, TAN> state;
};

template <int KD, int NW, Pass PASS, bool REV, bool TAN>
__device__ __forceinline__ void walk_or_state(const LinArgs& a, Storage<KD, NW, PASS, TAN>& sh,
                                              const Block& b) {
  if constexpr (PASS != kWalk) {
    if (PASS == kState || b.x.seg > 0)
      return walk<KD, NW, false, REV, TAN>(a, sh.state, b.x, b.u, b.head, b.vb0, b.part_at);
  }
  if constexpr (PASS != kState)
    walk<KD, NW, true, REV, TAN>(a, sh.main, b.x, b.u, b.head, b.vb0, b.part_at);
}

// One block of a launch of n walks.
template <int KD, int NW, Pass PASS>
__device__ __forceinline__ void mm_block(const LinWalks& ws, int n, Storage<KD, NW, PASS, false>& sh,
                                         uint32_t vblocks, uint32_t block, Places at) {
  const uint32_t r = block / (uint32_t)n;
  const LinArgs& a = ws.a[block - r * (uint32_t)n];
  if (r >= at.count * (uint32_t)a.heads * vblocks) return;
  const Block b = block_of<16 * NW>(a, r, vblocks, at.first);
  if (!b.on || (PASS == kWalk && a.lead && b.x.seg == 0)) return;
  if (a.rev)
    walk_or_state<KD, NW, PASS, true, false>(a, sh, b);
  else
    walk_or_state<KD, NW, PASS, false, false>(a, sh, b);
}
template <int KD, int NW, Pass PASS>
__device__ __forceinline__ void tan_block(const LinArgs& a, Storage<KD, NW, PASS, true>& sh,
                                          uint32_t vblocks, uint32_t r, Places at) {
  if (r >= at.count * (uint32_t)a.heads * vblocks) return;
  const Block b = block_of<16 * NW>(a, r, vblocks, at.first);
  // by the walks' launch alone: the states' may have other blocks and parts
  if (PASS == kWalk && !b.on && threadIdx.x == 0) a.dg_part[b.part_at] = 0.0f;
  if (!b.on || (PASS == kWalk && a.lead && b.x.seg == 0)) return;
  walk_or_state<KD, NW, PASS, false, true>(a, sh, b);
}

template <int KD, int NW, Pass PASS>
__global__ __launch_bounds__(64 * NW, waves_per_simd(KD, NW, PASS == kState, false)) void linattn_mm_kernel(
    LinWalks ws, uint32_t vblocks, Places at, uint32_t group) {
  __shared__ Storage<KD, NW, PASS, false> sh;
  mm_block<KD, NW, PASS>(ws, ws.n, sh, vblocks, xcd_block(blockIdx.x, group), at);
}

template <int KD, int NW, Pass PASS>
__global__ __launch_bounds__(64 * NW, waves_per_simd(KD, NW, PASS == kState, true)) void linattn_tan_kernel(
    LinArgs a, uint32_t vblocks, Places at, uint32_t group) {
  __shared__ Storage<KD, NW, PASS, true> sh;
  tan_block<KD, NW, PASS>(a, sh, vblocks, xcd_block(blockIdx.x, group), at);
}

// The walk with the derivative (the last of ws) and the others in one launch,
// its blocks first: they take longest, and side by side the two kinds fill the
// latencies of each other.  For heads of at most 64, three blocks to a CU either
// way: 192 x 2048 tokens of 64 take 214 us, in two launches 175 + 159.  (One
// register of the walks' launch is spilled.)  The derivative's block at heads of
// 128 holds a CU's registers alone.
constexpr bool beside(int kd, int nw) { return kd <= 64 && nw == 4; }

template <int KD, int NW, Pass PASS>
__global__ __launch_bounds__(64 * NW, 3) void linattn_beside_kernel(LinWalks ws, uint32_t vblocks,
                                                                    Places at, uint32_t group,
                                                                    uint32_t tan_group,
                                                                    uint32_t tan_grid) {
  __shared__ union {
    Storage<KD, NW, PASS, true> tan;
    Storage<KD, NW, PASS, false> mm;
  } sh;
  if (blockIdx.x < tan_grid)
    tan_block<KD, NW, PASS>(ws.a[ws.n - 1], sh.tan, vblocks, xcd_block(blockIdx.x, tan_group), at);
  else
    mm_block<KD, NW, PASS>(ws, ws.n - 1, sh.mm, vblocks, xcd_block(blockIdx.x - tan_grid, group),
                            at);
}

// Replaces the end states of the segments, the first one's and the others' own,
// by the states entering them: four state elements per thread, the segments of a
// sequence in order.  T likewise (X entering: Y <- a^n (Y + n X) + its own).
__global__ __launch_bounds__(256) void linattn_carry_kernel(LinWalks ws) {
  const LinArgs& a = ws.a[blockIdx.z];
  const int64_t per = (int64_t)a.heads * a.vd * a.kd;  // state elements of a sequence
  const int64_t e = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (e >= per) return;
  const int head = (int)(e / ((int64_t)a.vd * a.kd));
  for (int64_t seq = blockIdx.y; seq < a.nseq; seq += gridDim.y) {
    int first, len;
    sequence_of(a, (int)seq, first, len);
    const int segs = segments_of(a, len);
    if (segs == 1) continue;
    const int seg_len = segment_len(a, len);
    const Decays all = decays(a.log_decay[head], seg_len);
    const int64_t u0 = a.cu ? a.unit_table[1 + 2 * a.units + seq] : seq * a.segs;
    if (u0 >= a.units) continue;
    auto state = [&](float* ws_, int64_t k) {
      return reinterpret_cast<f32x4_t*>(ws_ + (u0 + k) * per + e);
    };
    f32x4_t X = *state(a.ws_state, 0), Y{0, 0, 0, 0};
    if (a.dg_part) Y = *state(a.ws_tangent, 0);
    for (int64_t k = 1; k < segs && u0 + k < a.units; ++k) {
      const float an = decay_of(all, (int)k - 1);
      f32x4_t* p = state(a.ws_state, k);
      const f32x4_t own = k + 1 < segs ? *p : f32x4_t{0, 0, 0, 0};
      *p = X;
      if (a.dg_part) {
        f32x4_t* q = state(a.ws_tangent, k);
        const f32x4_t mine = k + 1 < segs ? *q : f32x4_t{0, 0, 0, 0};
        *q = Y;
        Y = an * (Y + (float)seg_len * X) + mine;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) X[j] = __builtin_fmaf(an, X[j], own[j]);
    }
  }
}

// Waves of a block, 16 value channels each.  Four when 64 channels are enough,
// and where eight would not hold the derivative's walk in their registers.
int block_waves(int kd, int vd, bool tan) { return vd <= 64 || (tan && kd > 128) ? 4 : 8; }

// Blocks in runs of `group` that share an L2, and a grid of whole rounds.
struct Grid {
  uint32_t group, grid;
};
Grid grid_of(const LinArgs& a, uint32_t vblocks, Places at, uint32_t n) {
  const uint32_t blocks = at.count * (uint32_t)a.heads * vblocks * n;
  const uint32_t group =
      std::min((uint32_t)std::max({a.q.hdiv, a.k.hdiv, a.v.hdiv}) * vblocks * n, kMaxGroup);
  return {group, (blocks + 8 * group - 1) / (8 * group) * (8 * group)};
}

template <int KD, int NW, Pass PASS>
hipError_t launch_places(const LinWalks& ws, uint32_t vblocks, Places at, hipStream_t stream) {
  const LinArgs& last = ws.a[ws.n - 1];
  const dim3 threads(64 * NW);
  if (!last.dg_part) {
    const Grid m = grid_of(last, vblocks, at, (uint32_t)ws.n);
    hipLaunchKernelGGL((linattn_mm_kernel<KD, NW, PASS>), dim3(m.grid), threads, 0, stream, ws,
                       vblocks, at, m.group);
    return hipGetLastError();
  }
  const Grid t = grid_of(last, vblocks, at, 1);
  if constexpr (beside(KD, NW)) {
    if (ws.n > 1) {
      const Grid m = grid_of(last, vblocks, at, (uint32_t)ws.n - 1);
      hipLaunchKernelGGL((linattn_beside_kernel<KD, NW, PASS>), dim3(t.grid + m.grid), threads, 0,
                         stream, ws, vblocks, at, m.group, t.group, t.grid);
      return hipGetLastError();
    }
  }
  // alone: never in the lead, what goes beside only for its states, and 8 waves
  // never hold the derivative over 256 keys
  if constexpr (PASS != kLead && (PASS == kState || !beside(KD, NW)) && (KD <= 128 || NW == 4))
    hipLaunchKernelGGL((linattn_tan_kernel<KD, NW, PASS>), dim3(t.grid), threads, 0, stream, last,
                       vblocks, at, t.group);
  return hipGetLastError();
}

template <int KD, int NW, Pass PASS>
hipError_t launch_pass(const LinWalks& ws, hipStream_t stream) {
  const LinArgs& last = ws.a[ws.n - 1];
  const uint32_t vblocks = (uint32_t)((last.vd + 16 * NW - 1) / (16 * NW));
  const Places all = places_of(last, PASS);
  const uint32_t per = (uint32_t)last.heads * vblocks * (uint32_t)ws.n;  // blocks of a place
  for (uint32_t done = 0; done < all.count;) {
    const Places at = slice_of(all, done, 64 * NW, per, 2 * 8 * kMaxGroup);
    const hipError_t e = launch_places<KD, NW, PASS>(ws, vblocks, at, stream);
    if (e != hipSuccess) return e;
    done += at.count;
  }
  return hipSuccess;
}

template <int KD, int NW> hipError_t launch_walks(const LinWalks& ws, hipStream_t stream) {
  if (ws.a[0].seg_len) {
    // 4 waves for states alone: such blocks are half as long and spread better,
    // 32 heads of 128 over 32768 tokens in 4 segments 747 -> 677 us
    hipError_t e = ws.a[0].lead ? launch_pass<KD, NW, kLead>(ws, stream)
                                : launch_pass<KD, 4, kState>(ws, stream);
    if (e == hipSuccess && !ws.a[0].fold) e = launch_lin_carry(ws, stream);
    if (e != hipSuccess) return e;
  }
  return launch_pass<KD, NW, kWalk>(ws, stream);
}

template <int KD> hipError_t launch_kd(const LinWalks& ws, hipStream_t stream) {
  return block_waves(KD, ws.a[0].vd, ws.a[ws.n - 1].dg_part != nullptr) == 8
             ? launch_walks<KD, 8>(ws, stream)
             : launch_walks<KD, 4>(ws, stream);
}

}  // namespace

bool lin_decay_beside(int kd, int vd, bool io_bf16) {
  return io_bf16 && beside(kd, block_waves(kd, vd, true));
}

int64_t lin_dg_parts(int64_t units, int kd, int vd, bool io_bf16) {
  const int vb = 16 * (io_bf16 ? block_waves(kd, vd, true) : 4);
  return units * ((vd + vb - 1) / vb);
}

hipError_t launch_lin_carry(const LinWalks& ws, hipStream_t stream) {
  const LinArgs& a = ws.a[0];
  const int64_t per = (int64_t)a.heads * a.vd * a.kd / 4;
  const dim3 grid((unsigned)((per + 255) / 256), (unsigned)(a.nseq < 65535 ? a.nseq : 65535),
                  (unsigned)ws.n);
  hipLaunchKernelGGL(linattn_carry_kernel, grid, dim3(256), 0, stream, ws);
  return hipGetLastError();
}

hipError_t launch_lin_units(const LinArgs& a, hipStream_t stream) {
  if (!a.cu) return hipSuccess;
  hipLaunchKernelGGL(unit_table_kernel, dim3(1), dim3(kBuckets), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_linattn_mm(const LinArgs* walks, int n, hipStream_t stream) {
  LinWalks ws{};
  ws.n = n;
  for (int i = 0; i < n; ++i) ws.a[i] = walks[i];
  const int kd = walks[0].kd;
  if (kd <= 64) return launch_kd<64>(ws, stream);
  if (kd <= 128) return launch_kd<128>(ws, stream);
  return launch_kd<256>(ws, stream);
}

}  // namespace ssm
