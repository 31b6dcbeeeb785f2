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

  // (What a part leaves is taken by shift, mask and subtraction: the two-term dot
  // product does it in one, but runs on the matrix cores' path, 10 cycles among
  // their instructions, while these go beside them, two to each.)
  template <int N> __device__ __forceinline__ static Parts<N> split(const float* x) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = x[i];
    Parts<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      r.p[i] = last_parts(z);
      if (i + 1 < N) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[2 * j] -= part_lo(r.p[i][j]);
          z[2 * j + 1] -= part_hi(r.p[i][j]);
        }
      }
    }
    return r;
  }
  __device__ __forceinline__ static void unpack(const In& a, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = part_lo(a[i]), x[2 * i + 1] = part_hi(a[i]);
  }
  // A product in `steps` instructions: of two sums of parts those down to the last
  // part's size, the small ones first.
  static constexpr int steps(const In*, const In*) { return 1; }
  template <int N> static constexpr int steps(const In*, const Parts<N>*) { return N; }
  template <int N> static constexpr int steps(const Parts<N>*, const In*) { return N; }
  template <int N> static constexpr int steps(const Parts<N>*, const Parts<N>*) {
    return N * (N + 1) / 2;
  }
  __device__ __forceinline__ static f32x4_t step(const In& a, const In& b, f32x4_t c, int) {
    return mfma_k32(a, b, c);
  }
  template <int N>
  __device__ __forceinline__ static f32x4_t step(const In& a, const Parts<N>& b, f32x4_t c, int i) {
    return mfma_k32(a, b.p[N - 1 - i], c);
  }
  template <int N>
  __device__ __forceinline__ static f32x4_t step(const Parts<N>& a, const In& b, f32x4_t c, int i) {
    return mfma_k32(a.p[N - 1 - i], b, c);
  }
  template <int N>
  __device__ __forceinline__ static f32x4_t step(const Parts<N>& a, const Parts<N>& b, f32x4_t c,
                                                 int i) {
    // (a's last, b's first); (a's next, b's first two); ..
    int from = 0, n = 1;
    while (i >= from + n) from += n, ++n;
    return mfma_k32(a.p[N - n], b.p[n - 1 - (i - from)], c);
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
};

template <> struct Mat<float> {
  static constexpr int kParts = 1;
  struct In { f32x4_t lo, hi; };
  template <int N> struct Parts { f32x4_t lo, hi; };

  template <int N> __device__ __forceinline__ static Parts<N> split(const float* x) {
    return Parts<N>{{x[0], x[1], x[2], x[3]}, {x[4], x[5], x[6], x[7]}};
  }
  __device__ __forceinline__ static void unpack(const In& a, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a.lo[i], x[4 + i] = a.hi[i];
  }
  template <typename A, typename B> static constexpr int steps(const A*, const B*) { return 8; }
  template <typename A, typename B>
  __device__ __forceinline__ static f32x4_t step(const A& a, const B& b, f32x4_t c, int i) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(i < 4 ? a.lo[i & 3] : a.hi[i & 3],
                                                i < 4 ? b.lo[i & 3] : b.hi[i & 3], c, 0, 0, 0);
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
};

// c[n] += a[n] b, c[n] += a b[n], or c[n] += a[n] b[n]: a matrix instruction waits
// for the one before it on the same sum, and holds up the other wave's behind it, so
// the sums take turns.
template <typename M, int N, typename A, typename B>
__device__ __forceinline__ void mm(const A (&a)[N], const B& b, f32x4_t (&c)[N]) {
#pragma unroll
  for (int i = 0; i < M::steps((const A*)nullptr, (const B*)nullptr); ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) c[n] = M::step(a[n], b, c[n], i);
}
template <typename M, int N, typename A, typename B>
__device__ __forceinline__ void mm(const A& a, const B (&b)[N], f32x4_t (&c)[N]) {
#pragma unroll
  for (int i = 0; i < M::steps((const A*)nullptr, (const B*)nullptr); ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) c[n] = M::step(a, b[n], c[n], i);
}

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
  typedef Mat<IO> M;
  typedef typename M::In In;
  static constexpr int kPiece = 16 / sizeof(IO), kRow = W * sizeof(IO), kBytes = C * kRow;
  static constexpr int kPieces = W / kPiece;  // of a row

  // The exchange is linear in the bits of the row's number: address bits add up by
  // exclusive or where the numbers have no bit in common.
  __device__ __forceinline__ static constexpr int swap(int row) {
    return kPieces >= 16  ? ((row & 3) << 2) | ((row >> 2) & 3)
           : kPieces == 8 ? (((row >> 1) & 1) << 2) | ((row >> 2) & 3)
                          : (row >> 2) & (kPieces - 1);
  }
  __device__ __forceinline__ static int at(int row, int col) {  // byte address
    return row * kRow + ((col / kPiece) ^ swap(row)) * 16 + (col % kPiece) * (int)sizeof(IO);
  }
  // of (row + rows, col + 16-byte pieces), numbers without a bit in common
  __device__ __forceinline__ static int shift(int at, int rows, int pieces) {
    return (at ^ ((swap(rows) ^ pieces) * 16)) + rows * kRow;
  }

  // 8 columns from 32 ks + 8 g on of row r16 of the interleaved tile tt
  __device__ __forceinline__ static int rows_base(int r16, int g) { return at(row_of(0, r16), 8 * g); }
  __device__ __forceinline__ static In rows(const uint8_t* t, int base, int tt, int ks) {
    const int p = shift(base, 32 * (tt >> 1) + 4 * (tt & 1), ks * 32 / kPiece);
    if constexpr (sizeof(IO) == 2) {
      return *reinterpret_cast<const u32x4_t*>(t + p);
    } else {
      return {*reinterpret_cast<const f32x4_t*>(t + p), *reinterpret_cast<const f32x4_t*>(t + (p ^ 16))};
    }
  }

  // 8 rows from 32 p + 8 g on of a column: of column r16 of the interleaved tile kt
  // of 32 columns, or of column col0 + r16 (col0 a multiple of 16, kt 0)
  __device__ __forceinline__ static int keys_base(int r16, int g) {
    return sizeof(IO) == 2 ? at(8 * g + (r16 >> 2), 8 * (r16 & 3)) : at(8 * g, row_of(0, r16));
  }
  __device__ __forceinline__ static int cols_base(int r16, int g, int col0) {
    return sizeof(IO) == 2 ? at(8 * g + (r16 >> 2), col0 + 4 * (r16 & 3)) : at(8 * g, col0 + r16);
  }
  __device__ __forceinline__ static In cols(const uint8_t* t, int base, int p, int kt = 0) {
    if constexpr (sizeof(IO) == 2) {
      const int half = 8 * (kt & 1), over = 4 * (kt >> 1);
      return cat(lds_tr(t + shift(base, 32 * p, over) + half),
                 lds_tr(t + shift(base, 32 * p + 4, over) + half));
    } else {
      In x;
      const int over = 8 * (kt >> 1) + (kt & 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x.lo[j] = *reinterpret_cast<const float*>(t + shift(base, 32 * p + j, over));
        x.hi[j] = *reinterpret_cast<const float*>(t + shift(base, 32 * p + 4 + j, over));
      }
      return x;
    }
  }
  // 8 columns from col on of any row
  __device__ __forceinline__ static In row8(const uint8_t* t, int row, int col) {
    if constexpr (sizeof(IO) == 2) {
      return *reinterpret_cast<const u32x4_t*>(t + at(row, col));
    } else {
      return {*reinterpret_cast<const f32x4_t*>(t + at(row, col)),
              *reinterpret_cast<const f32x4_t*>(t + at(row, col + 4))};
    }
  }
};

// Which rows and columns the f-th fragment of a triangle holds (ssm_delta.h), and
// the other way round.
struct FragAt {
  int tt, ks;
};
template <bool UPPER> __device__ __forceinline__ FragAt frag_at(int f) {
  if (UPPER) return f < 4 ? FragAt{f >> 1, f & 1} : FragAt{f - 2, 1};
  return f < 4 ? FragAt{f, 0} : FragAt{f - 2, 1};
}
template <bool UPPER> __device__ __forceinline__ constexpr int frag_of(int tt, int ks) {
  return UPPER ? (tt < 2 ? 2 * tt + ks : tt + 2) : (ks == 0 ? tt : tt + 2);
}

// A [64, W] tile on its way into LDS: 16-byte pieces in the registers of THREADS
// threads.  Rows past n and columns past dim are zeros.
template <typename IO, int W, int THREADS> struct Loader {
  typedef Tile<IO, W> T;
  static constexpr int kPer = T::kPieces;
  static constexpr int kPasses = (C * kPer + THREADS - 1) / THREADS;
  static constexpr bool kAll = C * kPer % THREADS == 0;  // every thread has a piece each pass
  u32x4_t r[kPasses];

  __device__ __forceinline__ static int row(int p, int tid) { return (p * THREADS + tid) / kPer; }
  __device__ __forceinline__ static int col(int p, int tid) { return (tid % kPer) * T::kPiece; }
  __device__ __forceinline__ void load(const IO* base, int64_t stride, int n, int dim, int col0,
                                       int tid) {
    const uint32_t sb = (uint32_t)stride * (uint32_t)sizeof(IO);
    const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(
        base, n > 0 ? (uint32_t)(n - 1) * sb + (uint32_t)dim * (uint32_t)sizeof(IO) : 0u);
    // (a chunk's 64 rows span less than 2^30 bytes, so no offset wraps)
    const int c = col(0, tid) + col0;
    const uint32_t at = c < dim ? (uint32_t)(tid / kPer) * sb + (uint32_t)c * (uint32_t)sizeof(IO)
                                : 0x7f000000u;
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      r[p] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at + (uint32_t)(p * kRows) * sb, 0, 0));
  }
  // Where a thread's pieces stand: a pass takes whole rows, a power of two.
  static constexpr int kRows = THREADS / kPer;
  static_assert(THREADS % kPer == 0 && (kRows & (kRows - 1)) == 0, "whole rows a pass");
  __device__ __forceinline__ static int slot(int base, int p) { return T::shift(base, p * kRows, 0); }
  __device__ __forceinline__ static int slot_base(int tid) { return T::at(tid / kPer, col(0, tid)); }
  __device__ __forceinline__ void store(uint8_t* t, int tid) const {
    const int base = slot_base(tid);
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      if (kAll || row(p, tid) < C) *reinterpret_cast<u32x4_t*>(t + slot(base, p)) = r[p];
  }
  __device__ __forceinline__ bool odd() const {  // holds an infinity or a NaN
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

// The j-th of the n spans of a sequence; first: the number of its first span.
struct SpanAt {
  int seq, j, n, first;
};
__device__ __forceinline__ SpanAt spans_of_seq(const DeltaArgs& a, int seq) {
  if (!a.cu) return {seq, 0, a.per_spans, seq * a.per_spans};
  const int32_t* first = a.table + 2 * a.nseq + 1;
  return {seq, 0, first[seq + 1] - first[seq], first[seq]};
}
// of a span's number; seq < 0: there is no such span
__device__ __forceinline__ SpanAt span_at(const DeltaArgs& a, int span) {
  int seq;
  if (a.cu) {  // (every sequence has a span)
    const int32_t* first = a.table + 2 * a.nseq + 1;
    int lo = 0, hi = (int)a.nseq;
    if (span >= first[hi]) return {-1, 0, 0, 0};
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (first[mid] <= span) lo = mid;
      else hi = mid;
    }
    seq = lo;
  } else {
    seq = span / a.per_spans;
  }
  SpanAt s = spans_of_seq(a, seq);
  s.j = span - s.first;
  return s;
}

// The tokens t0 .. t0 + n - 1 of a chunk.
struct Chunk {
  int64_t t0;
  int n;
};
__device__ __forceinline__ Chunk chunk_of(const DeltaArgs& a, int64_t chunk) {
  int seq;
  if (a.cu) {  // the last sequence that begins at or before the chunk
    int lo = 0, hi = (int)a.nseq;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (a.table[mid] <= chunk) lo = mid;
      else hi = mid;
    }
    seq = lo;
  } else {
    seq = (int)(chunk / a.per);
  }
  const Seq s = seq_of(a, seq);
  const int c0 = (int)(chunk - s.chunk0) * C;
  return {(int64_t)s.first + c0, min(s.len - c0, C)};
}

}  // namespace
}  // namespace ssm
