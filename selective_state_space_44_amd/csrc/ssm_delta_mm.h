// ssm_delta_mm.h -- matrix products of the gated delta rule's kernels: operands of
// 16 x 16 tiles, tiles in LDS, sequences and chunks.
//
// A product of bf16 inputs runs on the bf16 matrix cores.  What is not bf16 by
// itself (states, solutions, weighted products) enters as a sum of bf16 parts: two
// keep 16 bits, three 24.  fp32 inputs run on the fp32 matrix instruction, whose
// products are exact to fp32.
//
// Both take the same operands: lane l holds row (or column) l % 16 and 8
// contraction slots 8 g + j, g = l / 16; the fp32 instruction takes the j-th slot
// of all four groups at a time.  A result tile has column l % 16 and rows 4 g + i.
// So that two result tiles are an operand of the next product, the rows of the
// tiles 2 p and 2 p + 1 are interleaved: row 4 g + i of either is row 32 p + 8 g +
// i (+ 4 in the second) of the matrix, and a lane holds rows 32 p + 8 g .. + 7.
#pragma once

#include "ssm_delta.h"
#include "ssm_mfma.h"

namespace ssm {
namespace {

constexpr int C = kDeltaChunk;

// Row of the matrix that row r of the interleaved tile t stands for.
__device__ __forceinline__ int row_of(int t, int r) {
  return 32 * (t >> 1) + 8 * (r >> 2) + (r & 3) + 4 * (t & 1);
}

template <typename IO> struct Mat;

template <> struct Mat<bf16> {
  static constexpr int kParts = 3;  // for fp32 accuracy
  typedef u32x4_t In;               // 8 inputs
  template <int N> struct Parts { u32x4_t p[N]; };

  __device__ __forceinline__ static In zero() { return u32x4_t{0, 0, 0, 0}; }
  template <int N> __device__ __forceinline__ static Parts<N> split(const float* x) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = x[i];
    Parts<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.p[i] = i + 1 < N ? take_parts(z) : last_parts(z);
    return r;
  }
  __device__ __forceinline__ static void unpack(const In& a, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = part_lo(a[i]), x[2 * i + 1] = part_hi(a[i]);
  }
  // c += a b; of two sums of parts, the products down to the last part's size
  __device__ __forceinline__ static f32x4_t mm(const In& a, const In& b, f32x4_t c) {
    return mfma_k32(a, b, c);
  }
  template <int N>
  __device__ __forceinline__ static f32x4_t mm(const In& a, const Parts<N>& b, f32x4_t c) {
#pragma unroll
    for (int i = N - 1; i >= 0; --i) c = mfma_k32(a, b.p[i], c);
    return c;
  }
  template <int N>
  __device__ __forceinline__ static f32x4_t mm(const Parts<N>& a, const In& b, f32x4_t c) {
#pragma unroll
    for (int i = N - 1; i >= 0; --i) c = mfma_k32(a.p[i], b, c);
    return c;
  }
  template <int N>
  __device__ __forceinline__ static f32x4_t mm(const Parts<N>& a, const Parts<N>& b, f32x4_t c) {
#pragma unroll
    for (int s = N - 1; s >= 0; --s)
#pragma unroll
      for (int i = 0; i <= s; ++i) c = mfma_k32(a.p[i], b.p[s - i], c);
    return c;
  }
  // the first N of more parts
  template <int N, int M> __device__ __forceinline__ static Parts<N> first(const Parts<M>& a) {
    Parts<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.p[i] = a.p[i];
    return r;
  }
  // bytes of 8 values as N parts, and access to a fragment [part][64 lanes] in LDS
  template <int N> static constexpr int kFragBytes = N * 1024;
  template <int N>
  __device__ __forceinline__ static void put(uint8_t* f, int lane, const Parts<N>& a) {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4_t*>(f + i * 1024 + lane * 16) = a.p[i];
  }
  template <int N> __device__ __forceinline__ static Parts<N> get(const uint8_t* f, int lane) {
    Parts<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.p[i] = *reinterpret_cast<const u32x4_t*>(f + i * 1024 + lane * 16);
    return r;
  }
  __device__ __forceinline__ static bool odd(const In& a) {  // holds an infinity or a NaN
    bool o = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o |= (a[i] & 0x7f800000u) == 0x7f800000u || (a[i] & 0x7f80u) == 0x7f80u;
    return o;
  }
};

template <> struct Mat<float> {
  static constexpr int kParts = 1;
  struct In { f32x4_t lo, hi; };
  template <int N> struct Parts { f32x4_t lo, hi; };

  __device__ __forceinline__ static In zero() { return In{{0, 0, 0, 0}, {0, 0, 0, 0}}; }
  template <int N> __device__ __forceinline__ static Parts<N> split(const float* x) {
    return Parts<N>{{x[0], x[1], x[2], x[3]}, {x[4], x[5], x[6], x[7]}};
  }
  __device__ __forceinline__ static void unpack(const In& a, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a.lo[i], x[4 + i] = a.hi[i];
  }
  template <typename A, typename B>
  __device__ __forceinline__ static f32x4_t mm(const A& a, const B& b, f32x4_t c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo[j], b.lo[j], c, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi[j], b.hi[j], c, 0, 0, 0);
    return c;
  }
  template <int N, int M> __device__ __forceinline__ static Parts<N> first(const Parts<M>& a) {
    return Parts<N>{a.lo, a.hi};
  }
  template <int N> static constexpr int kFragBytes = 2048;
  template <int N>
  __device__ __forceinline__ static void put(uint8_t* f, int lane, const Parts<N>& a) {
    *reinterpret_cast<f32x4_t*>(f + lane * 16) = a.lo;
    *reinterpret_cast<f32x4_t*>(f + 1024 + lane * 16) = a.hi;
  }
  template <int N> __device__ __forceinline__ static Parts<N> get(const uint8_t* f, int lane) {
    return Parts<N>{*reinterpret_cast<const f32x4_t*>(f + lane * 16),
                    *reinterpret_cast<const f32x4_t*>(f + 1024 + lane * 16)};
  }
  __device__ __forceinline__ static bool odd(const In& a) {
    bool o = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o |= (__float_as_uint(a.lo[i]) & 0x7f800000u) == 0x7f800000u ||
           (__float_as_uint(a.hi[i]) & 0x7f800000u) == 0x7f800000u;
    return o;
  }
};

// --- tiles in LDS ----------------------------------------------------------------
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// Transposing LDS read: in each group of 16 lanes, lane i gives the address of
// 4 consecutive elements (row i / 4, columns 4 (i % 4)..) and receives column
// i of the 4 rows.
__device__ __forceinline__ u32x2_t lds_tr(const uint8_t* p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// [64, W] elements, in 16-byte pieces; the pieces of a row are exchanged by its
// number so that what reads 8 rows of one piece (of consecutive rows, or of rows
// 0..3 and 8..11), and what reads 4 pieces of 4 consecutive rows, meets every bank
// once.
template <typename IO, int W> struct Tile {
  static constexpr int kPiece = 16 / sizeof(IO), kRow = W * sizeof(IO), kBytes = C * kRow;
  static constexpr int kPieces = W / kPiece;  // of a row

  __device__ __forceinline__ static int at(int row, int col) {  // byte address
    int f;
    if constexpr (kPieces >= 16) f = ((row & 3) << 2) | ((row >> 2) & 3);
    else if constexpr (kPieces == 8) f = (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
    else f = (row >> 2) & (kPieces - 1);
    const int piece = (col / kPiece) ^ f;
    return row * kRow + piece * 16 + (col % kPiece) * (int)sizeof(IO);
  }
  // 8 consecutive columns of a row
  __device__ __forceinline__ static typename Mat<IO>::In row8(const uint8_t* t, int row, int col) {
    if constexpr (sizeof(IO) == 2) {
      return *reinterpret_cast<const u32x4_t*>(t + at(row, col));
    } else {
      return {*reinterpret_cast<const f32x4_t*>(t + at(row, col)),
              *reinterpret_cast<const f32x4_t*>(t + at(row, col + 4))};
    }
  }
  // Rows 8 g' .. 8 g' + 7 (row8 = 8 g') of the lane's column: of `cols(c)`, the
  // column of lane c = l % 16.  The columns of lanes 4 i .. 4 i + 3 are
  // consecutive from a multiple of 4.
  template <typename F>
  __device__ __forceinline__ static typename Mat<IO>::In col8(const uint8_t* t, int row8, int r16,
                                                              F&& cols) {
    if constexpr (sizeof(IO) == 2) {
      const int c = cols(4 * (r16 & 3)), r = row8 + (r16 >> 2);
      return cat(lds_tr(t + at(r, c)), lds_tr(t + at(r + 4, c)));
    } else {
      typename Mat<IO>::In x;
      const int c = cols(r16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x.lo[j] = *reinterpret_cast<const float*>(t + at(row8 + j, c));
        x.hi[j] = *reinterpret_cast<const float*>(t + at(row8 + 4 + j, c));
      }
      return x;
    }
  }
};

// A [64, W] tile on its way into LDS: 16-byte pieces in the registers of THREADS
// threads.  Rows past n and columns past dim are zeros.
template <typename IO, int W, int THREADS> struct Loader {
  typedef Tile<IO, W> T;
  static constexpr int kPer = T::kPieces;
  static constexpr int kPasses = (C * kPer + THREADS - 1) / THREADS;
  static constexpr bool kAll = C * kPer % THREADS == 0;  // every thread has a piece each pass
  u32x4_t r[kPasses];

  __device__ __forceinline__ static int row(int p, int tid) { return (p * THREADS + tid) / kPer; }
  __device__ __forceinline__ static int col(int p, int tid) {
    return ((p * THREADS + tid) % kPer) * T::kPiece;
  }
  __device__ __forceinline__ void load(const IO* base, int64_t stride, int n, int dim, int col0,
                                       int tid) {
    const uint32_t sb = (uint32_t)stride * (uint32_t)sizeof(IO);
    const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(
        base, n > 0 ? (uint32_t)(n - 1) * sb + (uint32_t)dim * (uint32_t)sizeof(IO) : 0u);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int c = col(p, tid) + col0, i = row(p, tid);
      const uint32_t at = c < dim && (kAll || i < C)
                              ? (uint32_t)i * sb + (uint32_t)c * (uint32_t)sizeof(IO) : 0x7f000000u;
      r[p] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, 0));
    }
  }
  __device__ __forceinline__ void store(uint8_t* t, int tid) const {
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      if (kAll || row(p, tid) < C)
        *reinterpret_cast<u32x4_t*>(t + T::at(row(p, tid), col(p, tid))) = r[p];
  }
  __device__ __forceinline__ bool odd() const {
    bool o = false;
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o |= (r[p][i] & 0x7f800000u) == 0x7f800000u;
        if (sizeof(IO) == 2) o |= (r[p][i] & 0x7f80u) == 0x7f80u;
      }
    return o;
  }
};

// Block barrier that orders LDS only: loads of the next chunk and stores of
// results stay in flight over it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// --- sequences -------------------------------------------------------------------
struct Seq {
  int first, len;  // first token, number of tokens
  int chunk0;      // first chunk
  int chunks;
};

__device__ __forceinline__ int clamp_token(int t, int tokens) {
  return t < 0 ? 0 : t > tokens ? tokens : t;
}
__device__ __forceinline__ Seq seq_of(const DeltaArgs& a, int seq) {
  Seq s;
  if (!a.cu) {
    s.first = seq * (int)a.seqlen;
    s.len = (int)a.seqlen;
    s.chunk0 = seq * a.per;
    s.chunks = a.per;
    return s;
  }
  s.first = clamp_token(a.cu[seq], (int)a.tokens);
  const int end = clamp_token(a.cu[seq + 1], (int)a.tokens);
  s.len = end > s.first ? end - s.first : 0;
  s.chunk0 = a.table[seq];
  s.chunks = a.table[seq + 1] - s.chunk0;  // fewer where the table is full
  return s;
}

}  // namespace
}  // namespace ssm
