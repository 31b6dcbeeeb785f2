// ssm_norm.hip -- layer norm of rows and its gradients (gfx950, wave64).
//
//   h = (x - mean) r,  r = 1 / sqrt(mean((x - mean)^2) + eps),  y = h w + b;
// with g = dy w, per row and over the rows
//   dx = r (g - mean(g) - h mean(g h)),   dw = sum of dy h,   db = sum of dy.
//
// Bound by HBM: 16384 rows of 5120 channels in bf16 take 64 us forward (5.3 TB/s of
// the 336 MB that it has to read and write) and 105 backward (4.8 of 503 MB, the sums
// of dw and db included), where a large copy reaches 5.0.  A row is read once and
// stays in registers between its sums (the mean first, the squares around it after: rows
// far from zero lose nothing but the mean's own rounding, 2^-24 or so of its size).  A row
// belongs to a few lanes of a wave, to a wave, or to 4, 8 or 16 waves, whichever holds it
// in at most 32 channels a lane;
// blocks walk over many rows, so that weight and bias stay in registers as well, and
// ask for the next row before they reduce this one.  The backward's lanes add up dw
// and db of their channels in registers; the block's sums go to memory and a second
// launch adds them, every sum in a fixed order.
//
// Rows need no alignment: a lane's 16 bytes are read wherever they begin, and the last
// piece of a row that is not whole pieces is its last 16 bytes, whose first channels are
// the lane's before as well: both compute and store the same values, and the sums leave
// them out once (16384 rows of 5119 channels in bf16 84 us and 136 backward, of 5118 64
// and 107; with the last piece element by element 133 and 241).
#include <algorithm>

#include "ssm_device.h"
#include "ssm_norm.h"

namespace ssm {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// 16 bytes of a row.
template <typename IO> struct Piece {
  static constexpr int V = 16 / sizeof(IO);
  struct __attribute__((packed, aligned(sizeof(IO)))) Raw { u32x4_t v; };
  u32x4_t r;

  __device__ __forceinline__ void load(const IO* p) { r = reinterpret_cast<const Raw*>(p)->v; }
  __device__ __forceinline__ void store(IO* p) const { reinterpret_cast<Raw*>(p)->v = r; }
  // of fewer channels, the others zeros
  __device__ __forceinline__ void load(const IO* p, int n) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < n ? io<IO>::load(p + i) : 0.0f;
    pack(x);
  }
  __device__ __forceinline__ void store(IO* p, int n) const {
    float x[V];
    unpack(x);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) io<IO>::store(p + i, x[i]);
  }
  __device__ __forceinline__ void unpack(float* x) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (V == 4) {
        x[i] = __uint_as_float(r[i]);
      } else {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void pack(const float* x) {  // rounds to nearest even
    typedef __bf16 B2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (V == 4) {
        r[i] = __float_as_uint(x[i]);
      } else {
        const B2 b = {(__bf16)x[2 * i], (__bf16)x[2 * i + 1]};
        r[i] = __builtin_bit_cast(uint32_t, b);
      }
    }
  }
};

template <int CTRL> __device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// The sum over n = 1, 2, 4 .. 64 consecutive lanes, in all of them.
__device__ __forceinline__ float lane_sum(float v, int n) {
  if (n > 1) v += dpp<0xB1>(v);   // neighbours
  if (n > 2) v += dpp<0x4E>(v);   // pairs of a quad
  if (n > 4) v += dpp<0x141>(v);  // mirrored halves of 8
  if (n > 8) v += dpp<0x140>(v);  // mirrored halves of 16
  if (n > 16) v += __shfl_xor(v, 16);
  if (n > 32) v += __shfl_xor(v, 32);
  return v;
}

// Sums over a row's lanes: `lanes` of one wave, or the block's W waves.
template <int W> struct RowSum {
  float2 (*slot)[W];  // two, used in turn: one barrier a sum
  int turn = 0;
  __device__ __forceinline__ float2 operator()(float2 v, int lanes) {
    v.x = lane_sum(v.x, lanes);
    v.y = lane_sum(v.y, lanes);
    if constexpr (W > 1) {
      float2* s = slot[turn];
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
      __syncthreads();
      v = s[0];
#pragma unroll
      for (int w = 1; w < W; ++w) v.x += s[w].x, v.y += s[w].y;
    }
    return v;
  }
};

constexpr int threads_of(int w) { return w > 4 ? 64 * w : 256; }

// How rows end: with a whole piece, with one that begins before its place, or (kShort)
// within their only piece.
enum End { kWhole, kOver, kShort };

// The channels of a lane: pieces at (lane + f * lanes of the row) * V.
template <typename IO, int F, int W, End END> struct Row {
  typedef Piece<IO> P;
  static constexpr int V = P::V, E = V * F, T = threads_of(W);
  static constexpr End kEnd = END;
  int lanes;            // of a wave that share a row
  int c0, step, dim;    // first channel, channels between pieces, all
  int64_t row, stride;  // of the group's rows
  __device__ __forceinline__ Row(int lanes_, int dim_, uint32_t blocks) : lanes(lanes_), dim(dim_) {
    const int group = W > 1 ? 0 : threadIdx.x / lanes, groups = W > 1 ? 1 : T / lanes;
    const int lane = W > 1 ? threadIdx.x : threadIdx.x & (lanes - 1);
    c0 = lane * V;
    step = (W > 1 ? T : lanes) * V;
    row = (int64_t)blockIdx.x * groups + group;
    stride = (int64_t)blocks * groups;
  }
  __device__ __forceinline__ bool has(int f) const { return c0 + f * step < dim; }
  // its first channel, and how many of its channels are the piece's before
  __device__ __forceinline__ int at(int f) const {
    const int c = c0 + f * step;
    return END == kOver ? min(c, dim - V) : c;
  }
  __device__ __forceinline__ int over(int f) const { return END == kOver ? max(c0 + f * step + V - dim, 0) : 0; }
  // whether element i is of the row and counts
  __device__ __forceinline__ bool counts(int i) const {
    if (END == kOver) return i % V >= over(i / V);  // (beyond the row: over by V and more)
    return c0 + i / V * step + (END == kShort ? i % V : 0) < dim;
  }
  __device__ __forceinline__ int channel(int i) const { return at(i / V) + i % V; }
  __device__ __forceinline__ bool in(int i) const { return END == kShort ? counts(i) : has(i / V); }
  __device__ __forceinline__ void load(P& p, const IO* x, int f) const {
    p.r = u32x4_t{0, 0, 0, 0};
    if (END == kShort) p.load(x, dim);
    else if (has(f)) p.load(x + at(f));
  }
  __device__ __forceinline__ void store(const P& p, IO* x, int f) const {
    if (END == kShort) p.store(x, dim);
    else if (has(f)) p.store(x + at(f));
  }
};

// A lane's channels of weight or bias.
template <typename R> __device__ __forceinline__ void load_weight(const R& r, const float* w, float none,
                                                                  float* out) {
  typedef Piece<float> P;
#pragma unroll
  for (int i = 0; i < R::E; ++i) out[i] = none;
  if (!w) return;
  if constexpr (R::kEnd == kShort) {
#pragma unroll
    for (int i = 0; i < R::E; ++i)
      if (r.in(i)) out[i] = w[r.channel(i)];
  } else {
#pragma unroll
    for (int i = 0; i < R::E; i += P::V)
      if (r.in(i)) {
        P p;
        p.load(w + r.channel(i));
        p.unpack(out + i);
      }
  }
}

template <typename IO, int F, int W, End END>
__global__ __launch_bounds__(threads_of(W)) void norm_fwd_kernel(NormArgs a, int lanes) {
  typedef Row<IO, F, W, END> R;
  constexpr int V = R::V, E = R::E;
  __shared__ float2 sums[2][W];
  R r(lanes, a.dim, gridDim.x);
  RowSum<W> sum{sums};
  const int dim = a.dim;
  const float inv = 1.0f / (float)dim;
  const IO* x = static_cast<const IO*>(a.x);
  IO* y = static_cast<IO*>(a.out);
  Piece<IO> next[F];
  auto ask = [&](int64_t row) {
    if (row >= a.rows) return;
#pragma unroll
    for (int f = 0; f < F; ++f) r.load(next[f], x + row * a.x_stride, f);
  };
  ask(r.row);  // (first: its sums need neither weight nor bias)
  float w[E], b[E];
  load_weight(r, a.w, 1.0f, w);
  load_weight(r, a.b, 0.0f, b);
  // (groups of a block of one wave to a row end apart: they share no barrier)
  for (int64_t row = r.row; row < a.rows; row += r.stride) {
    float v[E];
#pragma unroll
    for (int f = 0; f < F; ++f) next[f].unpack(v + f * V);
    ask(row + r.stride);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += END != kOver || r.counts(i) ? v[i] : 0.0f;
    const float mean = sum(float2{s, 0.0f}, lanes).x * inv;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      v[i] -= mean;
      s = r.counts(i) ? __builtin_fmaf(v[i], v[i], s) : s;
    }
    const float rs = rsqrtf(__builtin_fmaf(sum(float2{s, 0.0f}, lanes).x, inv, a.eps));
#pragma unroll
    for (int f = 0; f < F; ++f) {
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i)
        o[i] = __builtin_fmaf(v[f * V + i] * rs, w[f * V + i], b[f * V + i]);
      Piece<IO> p;
      p.pack(o);
      r.store(p, y + row * dim, f);
    }
  }
}

template <typename IO, int F, int W, End END>
__global__ __launch_bounds__(threads_of(W)) void norm_bwd_kernel(NormArgs a, int lanes) {
  typedef Row<IO, F, W, END> R;
  constexpr int V = R::V, E = R::E;
  __shared__ float2 sums[2][W];
  R r(lanes, a.dim, gridDim.x);
  RowSum<W> sum{sums};
  const int dim = a.dim;
  const float inv = 1.0f / (float)dim;
  float w[E], dw[E], db[E];
  load_weight(r, a.w, 1.0f, w);
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.0f;
  const IO *x = static_cast<const IO*>(a.x), *dy = static_cast<const IO*>(a.dy);
  IO* dx = static_cast<IO*>(a.out);
  Piece<IO> xn[F], gn[F];
  auto ask = [&](int64_t row) {
    if (row >= a.rows) return;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      r.load(xn[f], x + row * a.x_stride, f);
      r.load(gn[f], dy + row * a.dy_stride, f);
    }
  };
  constexpr bool AHEAD = F < 8 || W < 8;  // (16384 channels in fp32: no registers for the next row)
  if (AHEAD) ask(r.row);
  for (int64_t row = r.row; row < a.rows; row += r.stride) {
    float v[E], g[E];
    if (!AHEAD) ask(row);
    float2 s{0.0f, 0.0f};
#pragma unroll
    for (int f = 0; f < F; ++f) {
      xn[f].unpack(v + f * V);
      gn[f].unpack(g + f * V);
    }
    if (AHEAD) ask(row + r.stride);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const bool on = END != kOver || r.counts(i);  // (elsewhere what is not there is zero)
      s.x += on ? v[i] : 0.0f;
      s.y = on ? __builtin_fmaf(g[i], w[i], s.y) : s.y;
    }
    s = sum(s, lanes);
    const float mean = s.x * inv, mg = s.y * inv;
    s = float2{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const bool on = r.counts(i);
      v[i] -= mean;
      s.x = on ? __builtin_fmaf(v[i], v[i], s.x) : s.x;
      s.y = on ? __builtin_fmaf(g[i] * w[i], v[i], s.y) : s.y;
    }
    s = sum(s, lanes);
    const float rs = rsqrtf(__builtin_fmaf(s.x, inv, a.eps)), mgh = s.y * inv * rs;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = f * V + i;
        const float h = v[e] * rs;
        dw[e] = __builtin_fmaf(g[e], h, dw[e]);
        db[e] += g[e];
        o[i] = rs * (__builtin_fmaf(g[e], w[e], -mg) - h * mgh);
      }
      Piece<IO> p;
      p.pack(o);
      r.store(p, dx + row * dim, f);
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * dim;
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = r.channel(i);
      if (r.in(i)) part[c] = dw[i], part[dim + c] = db[i];
    }
  } else {  // the block's groups, in order
    extern __shared__ float both[];  // [groups, dim]
    const int group = threadIdx.x / lanes, groups = R::T / lanes;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      if (pass) __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (r.in(i)) both[group * dim + r.channel(i)] = pass ? db[i] : dw[i];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < dim; c += R::T) {
        float t = 0.0f;
        for (int i = 0; i < groups; ++i) t += both[i * dim + c];
        part[pass * dim + c] = t;
      }
    }
  }
}

// dw, db: the sums over the blocks' parts; 32 threads to a channel, each every
// 32nd block, added in order.
__global__ __launch_bounds__(1024) void norm_parts_kernel(NormArgs a, int blocks) {
  __shared__ float part[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), i = threadIdx.x >> 5;
  float* out = blockIdx.y ? a.db : a.dw;
  if (!out) return;
  float s = 0.0f;
  if (col < a.dim) {
    const float* p = a.part + blockIdx.y * (int64_t)a.dim + col;
#pragma unroll 8
    for (int b = i; b < blocks; b += 32) s += p[(int64_t)b * 2 * a.dim];
  }
  part[i][threadIdx.x & 31] = s;
  __syncthreads();
  if (i == 0 && col < a.dim) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += part[k][threadIdx.x & 31];
    out[col] = t;
  }
}

// How a row lies: lanes of a wave that share it, and rows of a block.
struct Shape {
  int waves, pieces, lanes, groups;
};
Shape shape_of(int dim, bool bf16, bool bwd) {
  const int v = bf16 ? 8 : 4, pieces = (dim + v - 1) / v;
  if (pieces <= 256) {  // a wave, or less
    int lanes = 1;
    while (lanes < pieces && lanes < 64) lanes *= 2;
    const int f = (pieces + lanes - 1) / lanes;
    return {1, f > 2 ? 4 : f, lanes, 256 / lanes};
  }
  int f = (pieces + 255) / 256;
  if (f <= (bf16 ? 4 : 8)) return {4, bf16 ? f : (f + 1) / 2 * 2, 64, 1};
  // 16 waves have 128 registers each: the backward, which holds twice as much, takes 8
  // (4096 rows of 16384 channels in bf16: 226 us with 16, 106 with 8)
  if (!bwd) return {16, bf16 ? 2 : 4, 64, 1};
  f = (pieces + 511) / 512;
  return {8, bf16 ? f : (f + 1) / 2 * 2, 64, 1};
}

// Blocks: as many as the CUs hold at once, three of four waves and in the backward
// two, so that all walk over as many rows and none begins late.  Of 512, 768, 1024 and
// 1280 blocks forward, bf16: 16384 rows of 5120 74, 64, 66 and 75 us; wide ones 128, 256
// and 512 4096 of 16384 81, 49 and 51.  Of 256, 512 and 768 backward, whose blocks write
// their sums besides: 16384 of 5120 139, 105 and 135 us, 65536 of 1024 117, 79 and 84.
constexpr int kFwdBlocks = 768, kBwdBlocks = 512, kWideBlocks = 256;
// A group's rows backward, four at least where that leaves 128 blocks (64 rows of 4096
// channels 10.7 us in blocks of a row, 14.8 of four; 600 of 5120 29.0 and 20.7).
constexpr int kBwdRows = 4, kBwdFew = 128;

template <typename IO, int F, int W, End END, bool BWD>
hipError_t launch_t(const NormArgs& a, const Shape& s, hipStream_t stream) {
  if constexpr (BWD) {
    const int blocks = norm_bwd_blocks(a.rows, a.dim, sizeof(IO) == 2);
    const size_t lds = W == 1 && a.part ? (size_t)s.groups * a.dim * 4 : 0;
    hipLaunchKernelGGL((norm_bwd_kernel<IO, F, W, END>), dim3(blocks), dim3(threads_of(W)), lds,
                       stream, a, s.lanes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    hipLaunchKernelGGL(norm_parts_kernel, dim3((a.dim + 31) / 32, 2), dim3(1024), 0, stream, a,
                       blocks);
  } else {
    const int64_t want = (a.rows + s.groups - 1) / s.groups;
    const int blocks = (int)std::min<int64_t>(want, W > 4 ? kWideBlocks : kFwdBlocks);
    hipLaunchKernelGGL((norm_fwd_kernel<IO, F, W, END>), dim3(blocks), dim3(threads_of(W)), 0,
                       stream, a, s.lanes);
  }
  return hipGetLastError();
}
template <typename IO, int F, int W, bool BWD>
hipError_t launch_f(const NormArgs& a, const Shape& s, hipStream_t stream) {
  if constexpr (F == 1 && W == 1)
    if (a.dim < Piece<IO>::V) return launch_t<IO, F, W, kShort, BWD>(a, s, stream);
  return a.dim % Piece<IO>::V ? launch_t<IO, F, W, kOver, BWD>(a, s, stream)
                              : launch_t<IO, F, W, kWhole, BWD>(a, s, stream);
}
template <bool BWD> hipError_t launch(const NormArgs& a, bool bf, hipStream_t stream) {
  const Shape s = shape_of(a.dim, bf, BWD);
  switch (s.waves * 100 + s.pieces) {
    case 101: return bf ? launch_f<bf16, 1, 1, BWD>(a, s, stream) : launch_f<float, 1, 1, BWD>(a, s, stream);
    case 102: return bf ? launch_f<bf16, 2, 1, BWD>(a, s, stream) : launch_f<float, 2, 1, BWD>(a, s, stream);
    case 104: return bf ? launch_f<bf16, 4, 1, BWD>(a, s, stream) : launch_f<float, 4, 1, BWD>(a, s, stream);
    case 402: return bf ? launch_f<bf16, 2, 4, BWD>(a, s, stream) : launch_f<float, 2, 4, BWD>(a, s, stream);
    case 403: return launch_f<bf16, 3, 4, BWD>(a, s, stream);
    case 404: return bf ? launch_f<bf16, 4, 4, BWD>(a, s, stream) : launch_f<float, 4, 4, BWD>(a, s, stream);
    case 406: return launch_f<float, 6, 4, BWD>(a, s, stream);
    case 408: return launch_f<float, 8, 4, BWD>(a, s, stream);
  }
  if constexpr (BWD) {
    if (bf) return s.pieces == 3 ? launch_f<bf16, 3, 8, BWD>(a, s, stream) : launch_f<bf16, 4, 8, BWD>(a, s, stream);
    return s.pieces == 6 ? launch_f<float, 6, 8, BWD>(a, s, stream) : launch_f<float, 8, 8, BWD>(a, s, stream);
  } else {
    return bf ? launch_f<bf16, 2, 16, BWD>(a, s, stream) : launch_f<float, 4, 16, BWD>(a, s, stream);
  }
}

}  // namespace

int norm_bwd_blocks(int64_t rows, int dim, bool io_bf16) {
  const Shape s = shape_of(dim, io_bf16, true);
  const int64_t all = std::max<int64_t>((rows + s.groups - 1) / s.groups, 1);  // of a row to a group
  const int64_t want = std::max((all + kBwdRows - 1) / kBwdRows, std::min<int64_t>(all, kBwdFew));
  return (int)std::min<int64_t>(want, s.waves > 4 ? kWideBlocks : kBwdBlocks);
}

hipError_t launch_norm_fwd(const NormArgs& a, bool io_bf16, hipStream_t stream) {
  return launch<false>(a, io_bf16, stream);
}
hipError_t launch_norm_bwd(const NormArgs& a, bool io_bf16, hipStream_t stream) {
  return launch<true>(a, io_bf16, stream);
}

}  // namespace ssm
