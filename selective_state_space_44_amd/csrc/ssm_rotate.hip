// ssm_rotate.hip -- RMS norm of every query and key head with the position
// rotation in the same pass, and its gradients (gfx950, wave64).
//
// A head's row x [dim] becomes u = x * r * w with r = 1 / sqrt(mean(x^2) +
// eps), and the pairs of its first `rot` channels are turned by the angle of
// the token's position: (a, b) -> (a c - b s, a s + b c).  The transpose of a
// turn is the turn by the opposite angle, so with g = turned-back dy
//   dw = sum over rows of g * x * r,   dx = r * (w g - x r * mean(w g x r)).
//
// Bound by HBM: every channel is read and written once and nothing else is
// large, so the kernels keep a row in the registers of a few lanes.  Lane j of
// a row holds two vectors of V channels that form V pairs: channels jV.. and
// rot/2 + jV.. (or 2V consecutive channels when pairs are neighbours); the
// channels past `rot` are split in two halves the same way and turned by the
// angle 0.  So the turn needs no exchange between lanes, and the row's sum of
// squares is a few DPP steps.  Arithmetic is fp32; a bf16 result is rounded
// once.  Measured at 16384 tokens of 40 + 8 heads of 128 bf16, where a large
// copy reaches 4.9 TB/s: forward 79 us, 5.1 TB/s; backward with both weights'
// gradients 120 us, 5.0 TB/s; pairs side by side 82 and 135 us; fp32 146 and 232
// us, 5.5 and 5.2 TB/s.  A decode batch of 16 tokens takes as long as its
// launch.
#include <algorithm>

#include "ssm_device.h"
#include "ssm_linattn.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kBwdBlocks = 1024;  // four to a CU

template <typename IO, int V> struct Vec;
template <int V> struct Vec<float, V> {  // accesses of at most 16 bytes
  static constexpr int W = V < 4 ? V : 4;
  typedef float T __attribute__((ext_vector_type(W)));
  __device__ __forceinline__ static void load(const float* p, float* out) {
#pragma unroll
    for (int k = 0; k < V; k += W) {
      const T t = *reinterpret_cast<const T*>(p + k);
#pragma unroll
      for (int i = 0; i < W; ++i) out[k + i] = t[i];
    }
  }
  __device__ __forceinline__ static void store(float* p, const float* in) {
#pragma unroll
    for (int k = 0; k < V; k += W) {
      T t;
#pragma unroll
      for (int i = 0; i < W; ++i) t[i] = in[k + i];
      *reinterpret_cast<T*>(p + k) = t;
    }
  }
};
template <int V> struct Vec<bf16, V> {
  struct alignas(2 * V) T { uint32_t w[V / 2]; };
  __device__ __forceinline__ static void load(const bf16* p, float* out) {
    const T t = *reinterpret_cast<const T*>(p);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const uint32_t w = t.w[i];
      out[2 * i] = __uint_as_float(w << 16);
      out[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static void store(bf16* p, const float* in) {
    typedef __bf16 B2 __attribute__((ext_vector_type(2)));
    T t;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const B2 b = {(__bf16)in[2 * i], (__bf16)in[2 * i + 1]};  // round to nearest even
      t.w[i] = __builtin_bit_cast(uint32_t, b);
    }
    *reinterpret_cast<T*>(p) = t;
  }
};

template <int CTRL> __device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// The sum over the n = 1, 2, 4 .. 64 lanes of a row, in all of them.
__device__ __forceinline__ float row_sum(float v, int n) {
  if (n > 1) v += dpp<0xB1>(v);   // neighbours
  if (n > 2) v += dpp<0x4E>(v);   // pairs of a quad
  if (n > 4) v += dpp<0x141>(v);  // mirrored halves of 8
  if (n > 8) v += dpp<0x140>(v);  // mirrored halves of 16
  if (n > 16) v += __shfl_xor(v, 16);
  if (n > 32) v += __shfl_xor(v, 32);
  return v;
}

// What lane j of a row holds: the two vectors' channel offsets (INTER: one run
// of 2V channels at `a`), whether it holds any, and its pairs' table column.
struct Place {
  int a, b, col;
  bool on, turned;
};
template <int V, bool INTER>
__device__ __forceinline__ Place place_of(int j, int dim, int rot) {
  const int np = rot / (2 * V), rest = rot + (j - np) * V;
  const bool turned = j < np;
  const int at = INTER ? 2 * V * j : turned ? j * V : rest;
  const int past = INTER ? V : turned ? rot / 2 : (dim - rot) / 2;
  return {at, at + past, j * V, j < dim / (2 * V), turned};
}

// Cosines and sines of a token's pairs: of the angle 0 past rot, NaN for a
// position outside the table (no read outside it).
template <int V>
__device__ __forceinline__ void load_turn(const RotateArgs& a, uint32_t t, const Place& p,
                                          float* c, float* s) {
  int64_t pos = -1;
  if (p.turned) pos = a.positions ? a.positions[t] : (int64_t)(t % a.seqlen);
  const bool in = pos >= 0 && pos < a.npos;
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = 1.0f, s[i] = 0.0f;
  if (in) {
    const int64_t at = pos * (a.rot / 2) + p.col;
    Vec<float, V>::load(a.cos + at, c);
    Vec<float, V>::load(a.sin + at, s);
  }
  const bool nan = p.turned && !in;
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = nan ? __uint_as_float(0x7fc00000u) : c[i];
}

// x[0..V) and x[V..2V) are the pairs' halves, in either layout.
template <typename IO, int V, bool INTER>
__device__ __forceinline__ void load_pairs(const IO* row, const Place& p, float* x) {
  float t[2 * V];
  if (INTER) {
    Vec<IO, 2 * V>::load(row + p.a, t);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = t[2 * i], x[V + i] = t[2 * i + 1];
  } else {
    Vec<IO, V>::load(row + p.a, x);
    Vec<IO, V>::load(row + p.b, x + V);
  }
}
template <typename IO, int V, bool INTER>
__device__ __forceinline__ void store_pairs(IO* row, const Place& p, const float* x) {
  if (INTER) {
    float t[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[2 * i] = x[i], t[2 * i + 1] = x[V + i];
    Vec<IO, 2 * V>::store(row + p.a, t);
  } else {
    Vec<IO, V>::store(row + p.a, x);
    Vec<IO, V>::store(row + p.b, x + V);
  }
}

// One unit is up to U consecutive heads of q or of k of one token, handled by
// one group of `lanes` lanes: the heads share the token's cosines and sines.
__device__ __forceinline__ int units_per_token(int heads, int U) { return (heads + U - 1) / U; }

template <typename IO, int V, bool INTER, int U>
__global__ __launch_bounds__(kThreads) void rotate_fwd_kernel(RotateArgs a, int lanes,
                                                              uint32_t units, uint32_t block0) {
  const int j = threadIdx.x & (lanes - 1);
  const uint32_t unit = (block0 + blockIdx.x) * (uint32_t)(kThreads / lanes) + threadIdx.x / lanes;
  if (unit >= units) return;
  const uint32_t uq = units_per_token(a.heads[0], U), uk = units_per_token(a.heads[1], U);
  const uint32_t t = unit / (uq + uk);
  uint32_t first = unit - t * (uq + uk);
  const int which = first >= uq;
  if (which) first -= uq;
  const int h0 = first * U, n = a.heads[which] - h0;
  const Place p = place_of<V, INTER>(j, a.dim, a.rot);
  float x[U][2 * V];
  const IO* in = static_cast<const IO*>(a.x[which]) + t * a.stride[which] + h0 * a.dim;
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) x[u][i] = 0.0f;
    if (p.on && u < n) load_pairs<IO, V, INTER>(in + u * a.dim, p, x[u]);
  }
  float c[V], s[V], w[2 * V];
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) w[i] = 1.0f;
  load_turn<V>(a, t, p, c, s);
  if (p.on && a.w[which]) load_pairs<float, V, INTER>(a.w[which], p, w);
  IO* out = static_cast<IO*>(a.out[which]) + ((int64_t)t * a.heads[which] + h0) * a.dim;
  const float inv = 1.0f / (float)a.dim;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) ss = __builtin_fmaf(x[u][i], x[u][i], ss);
    const float r = rsqrtf(__builtin_fmaf(row_sum(ss, lanes), inv, a.eps));
    float y[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float ua = x[u][i] * r * w[i], ub = x[u][V + i] * r * w[V + i];
      y[i] = ua * c[i] - ub * s[i];
      y[V + i] = ua * s[i] + ub * c[i];
    }
    if (p.on && u < n) store_pairs<IO, V, INTER>(out + u * a.dim, p, y);
  }
}

// The backward's blocks: the first of them take q's rows, the others k's, in
// the proportion of their rows, so that a lane keeps one weight and one
// gradient in registers.  A group takes one row at a time: two rows at once
// share the cosines and sines but leave 3 waves to a SIMD in place of 4, 171 us
// against 131 at 16384 tokens, 40 + 8 heads of 128 bf16.
struct BwdBlocks {
  int q, k;
};

// The weights' gradients: every lane group sums its rows' g * x * r in
// registers, the block adds its groups in order into dw_part, and a second
// kernel adds the blocks in order, so that results repeat bit for bit.
template <typename IO, int V, bool INTER>
__global__ __launch_bounds__(kThreads) void rotate_bwd_kernel(RotateArgs a, int lanes,
                                                              BwdBlocks blocks) {
  const int j = threadIdx.x & (lanes - 1);
  const uint32_t groups = kThreads / lanes;
  const int which = (int)blockIdx.x >= blocks.q;
  const uint32_t block = which ? blockIdx.x - blocks.q : blockIdx.x;
  const uint32_t heads = which ? a.heads[1] : a.heads[0];
  const uint32_t rows = (uint32_t)a.tokens * heads;
  const int64_t stride = which ? a.stride[1] : a.stride[0];
  const int64_t dstride = which ? a.dstride[1] : a.dstride[0];
  const IO* in = static_cast<const IO*>(which ? a.x[1] : a.x[0]);
  const IO* dy = static_cast<const IO*>(which ? a.dy[1] : a.dy[0]);
  IO* out = static_cast<IO*>(which ? a.out[1] : a.out[0]);
  const float* weight = which ? a.w[1] : a.w[0];
  const uint32_t step = (which ? blocks.k : blocks.q) * groups;
  const Place p = place_of<V, INTER>(j, a.dim, a.rot);
  const float inv = 1.0f / (float)a.dim;
  float w[2 * V], acc[2 * V];
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) w[i] = 1.0f, acc[i] = 0.0f;
  if (p.on && weight) load_pairs<float, V, INTER>(weight, p, w);
  for (uint32_t row = block * groups + threadIdx.x / lanes; row < rows; row += step) {
    const uint32_t t = row / heads;
    const int at = (row - t * heads) * a.dim;
    float x[2 * V], g[2 * V];
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) x[i] = g[i] = 0.0f;
    float c[V], s[V];
    if (p.on) {
      load_pairs<IO, V, INTER>(in + t * stride + at, p, x);
      load_pairs<IO, V, INTER>(dy + t * dstride + at, p, g);
    }
    load_turn<V>(a, t, p, c, s);
    float ss = 0.0f, dot = 0.0f;
    float wg[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float ga = g[i], gb = g[V + i];
      g[i] = ga * c[i] + gb * s[i];
      g[V + i] = gb * c[i] - ga * s[i];
    }
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) {
      wg[i] = w[i] * g[i];
      ss = __builtin_fmaf(x[i], x[i], ss);
      dot = __builtin_fmaf(wg[i], x[i], dot);
    }
    ss = row_sum(ss, lanes);
    dot = row_sum(dot, lanes);
    const float r = rsqrtf(__builtin_fmaf(ss, inv, a.eps));
    const float k = dot * inv * r * r;  // mean(w g x r) * r
    float dx[2 * V];
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) {
      dx[i] = r * (wg[i] - x[i] * k);
      acc[i] = __builtin_fmaf(g[i] * r, x[i], acc[i]);
    }
    if (p.on) store_pairs<IO, V, INTER>(out + (int64_t)row * a.dim, p, dx);
  }
  if (!a.dw_part) return;
  extern __shared__ float part[];  // [groups, dim]
  float* mine = part + (threadIdx.x / lanes) * a.dim;
  if (p.on) store_pairs<float, V, INTER>(mine, p, acc);
  __syncthreads();
  for (int d = threadIdx.x; d < a.dim; d += kThreads) {
    float sum = 0.0f;
    for (uint32_t i = 0; i < groups; ++i) sum += part[i * a.dim + d];
    a.dw_part[(int64_t)blockIdx.x * a.dim + d] = sum;
  }
}

// dw[which][d] = sum over its blocks of part[block, d]; 64 threads to a
// channel, each a run of blocks, added in order.
__global__ __launch_bounds__(1024) void rotate_dw_kernel(RotateArgs a, BwdBlocks blocks) {
  __shared__ float part[64][17];
  const int col = blockIdx.x * 16 + (threadIdx.x & 15), row = threadIdx.x >> 4;
  const int which = blockIdx.y;
  if (!a.dw[which]) return;
  const int b0 = which ? blocks.q : 0, b1 = which ? blocks.q + blocks.k : blocks.q;
  float s = 0.0f;
  if (col < a.dim)
    for (int b = b0 + row; b < b1; b += 64) s += a.dw_part[(int64_t)b * a.dim + col];
  part[row][threadIdx.x & 15] = s;
  __syncthreads();
  if (row == 0 && col < a.dim) {
    float t = 0.0f;
    for (int i = 0; i < 64; ++i) t += part[i][threadIdx.x & 15];
    a.dw[which][col] = t;
  }
}

// Channels a lane holds per half: the widest vector that divides both the
// turned pairs and the rest.
int vec_of(const RotateArgs& a, int most) {
  for (int v = most; v > 2; v /= 2)
    if ((a.rot / 2) % v == 0 && ((a.dim - a.rot) / 2) % v == 0) return v;
  return 2;
}
int lanes_of(int dim, int v) {
  int n = 1;
  while (n * 2 * v < dim) n *= 2;
  return n;
}

template <typename IO, int V, bool INTER>
hipError_t fwd_v(const RotateArgs& a, hipStream_t stream) {
  const int lanes = lanes_of(a.dim, V);
  constexpr int U = 2;
  const uint32_t units =
      (uint32_t)a.tokens * ((a.heads[0] + U - 1) / U + (a.heads[1] + U - 1) / U);
  const uint32_t per = kThreads / lanes, blocks = (units + per - 1) / per;
  for (uint32_t b = 0; b < blocks; b += std::min(blocks - b, max_blocks(kThreads))) {
    hipLaunchKernelGGL((rotate_fwd_kernel<IO, V, INTER, U>),
                       dim3(std::min(blocks - b, max_blocks(kThreads))), dim3(kThreads), 0, stream,
                       a, lanes, units, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename IO, int V, bool INTER>
hipError_t bwd_v(const RotateArgs& a, hipStream_t stream) {
  const int lanes = lanes_of(a.dim, V), groups = kThreads / lanes;
  BwdBlocks blocks{0, 0};
  if (const int heads = a.heads[0] + a.heads[1]) {
    const int64_t total = rotate_bwd_blocks(a.tokens, heads, a.dim);
    blocks.k = (int)(total * a.heads[1] / heads);
    if (a.heads[1] > 0 && blocks.k == 0) blocks.k = 1;
    blocks.q = (int)total - blocks.k;
    hipLaunchKernelGGL((rotate_bwd_kernel<IO, V, INTER>), dim3((unsigned)total), dim3(kThreads),
                       (size_t)groups * a.dim * 4, stream, a, lanes, blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dw_part) return hipSuccess;
  hipLaunchKernelGGL(rotate_dw_kernel, dim3((a.dim + 15) / 16, 2), dim3(1024), 0, stream, a,
                     blocks);
  return hipGetLastError();
}

// At most 8 channels a half (16 bytes of bf16; 4 of fp32, and interleaved pairs
// are one run of 2V): with 4 for bf16 the backward takes 160 us in place of 131
// and the forward 96 in place of 87 at the size above.
template <typename IO, bool INTER, bool BWD>
hipError_t launch_i(const RotateArgs& a, hipStream_t stream) {
  constexpr int most = sizeof(IO) == 2 && !INTER ? 8 : 4;
  switch (vec_of(a, most)) {
    case 8:
      if constexpr (most == 8) return BWD ? bwd_v<IO, 8, INTER>(a, stream) : fwd_v<IO, 8, INTER>(a, stream);
    case 4: return BWD ? bwd_v<IO, 4, INTER>(a, stream) : fwd_v<IO, 4, INTER>(a, stream);
    default: return BWD ? bwd_v<IO, 2, INTER>(a, stream) : fwd_v<IO, 2, INTER>(a, stream);
  }
}
template <bool BWD> hipError_t launch(const RotateArgs& a, bool io_bf16, hipStream_t stream) {
  if (io_bf16)
    return a.interleaved ? launch_i<bf16, true, BWD>(a, stream) : launch_i<bf16, false, BWD>(a, stream);
  return a.interleaved ? launch_i<float, true, BWD>(a, stream) : launch_i<float, false, BWD>(a, stream);
}

}  // namespace

// Blocks of the backward: kBwdBlocks, fewer when there are not that many rows,
// but one for q and one for k.
int rotate_bwd_blocks(int64_t tokens, int heads, int dim) {
  const int64_t want = (tokens * heads * dim + 8191) / 8192;
  return (int)std::min<int64_t>(std::max<int64_t>(want, 2), kBwdBlocks);
}

hipError_t launch_rotate_fwd(const RotateArgs& a, bool io_bf16, hipStream_t stream) {
  return launch<false>(a, io_bf16, stream);
}
hipError_t launch_rotate_bwd(const RotateArgs& a, bool io_bf16, hipStream_t stream) {
  return launch<true>(a, io_bf16, stream);
}

}  // namespace ssm
