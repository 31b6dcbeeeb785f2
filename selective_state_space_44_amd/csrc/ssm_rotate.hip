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
// once.
#include "ssm_device.h"
#include "ssm_linattn.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

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

__device__ __forceinline__ float row_sum(float v, int n) {
  for (int m = 1; m < n; m <<= 1) v += __shfl_xor(v, m);
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
  Place p;
  const int np = rot / (2 * V);
  p.on = j < dim / (2 * V);
  p.turned = j < np;
  p.col = j * V;
  if (INTER) {
    p.a = 2 * V * j;
    p.b = p.a + V;
  } else if (p.turned) {
    p.a = j * V;
    p.b = rot / 2 + j * V;
  } else {
    p.a = rot + (j - np) * V;
    p.b = rot + (dim - rot) / 2 + (j - np) * V;
  }
  return p;
}

// Cosines and sines of a token's pairs (untouched past rot).  A position outside the table turns to NaN (no read outside it).
template <int V>
__device__ __forceinline__ void load_turn(const RotateArgs& a, int64_t t, const Place& p,
                                          float* c, float* s) {
  if (!p.turned) return;
  const int64_t pos = a.positions ? a.positions[t] : t % a.seqlen;
  if (pos < 0 || pos >= a.npos) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = s[i] = __uint_as_float(0x7fc00000u);
    return;
  }
  const int64_t at = pos * (a.rot / 2) + p.col;
  Vec<float, V>::load(a.cos + at, c);
  Vec<float, V>::load(a.sin + at, s);
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
// one group of `lanes` lanes.
template <int U>
__device__ __forceinline__ void unit_of(const RotateArgs& a, int64_t unit, int64_t& t, int& which,
                                        int& h0, int& n) {
  const int uq = (a.heads[0] + U - 1) / U, uk = (a.heads[1] + U - 1) / U;
  t = unit / (uq + uk);
  int u = (int)(unit - t * (uq + uk));
  which = u >= uq;
  if (which) u -= uq;
  h0 = u * U;
  n = a.heads[which] - h0 < U ? a.heads[which] - h0 : U;
}

template <typename IO, int V, bool INTER, int U>
__global__ __launch_bounds__(kThreads) void rotate_fwd_kernel(RotateArgs a, int lanes,
                                                              int64_t units) {
  const int j = threadIdx.x & (lanes - 1);
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / lanes;
  if (unit >= units) return;
  int64_t t;
  int which, h0, n;
  unit_of<U>(a, unit, t, which, h0, n);
  const Place p = place_of<V, INTER>(j, a.dim, a.rot);
  float x[U][2 * V];
  const IO* in = static_cast<const IO*>(a.x[which]) + t * a.stride[which] + (int64_t)h0 * a.dim;
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) x[u][i] = 0.0f;
    if (p.on && u < n) load_pairs<IO, V, INTER>(in + u * a.dim, p, x[u]);
  }
  float c[V], s[V], w[2 * V];
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) w[i] = 1.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = 1.0f, s[i] = 0.0f;
  if (p.on) {
    load_turn<V>(a, t, p, c, s);
    if (a.w[which]) load_pairs<float, V, INTER>(a.w[which], p, w);
  }
  IO* out = static_cast<IO*>(a.out[which]) + (t * a.heads[which] + h0) * a.dim;
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

// The weights' gradients: every lane group sums its rows' g * x * r in
// registers, the block adds its groups in order into dw_part, and a second
// kernel adds the blocks in order, so that results repeat bit for bit.
template <typename IO, int V, bool INTER, int U>
__global__ __launch_bounds__(kThreads) void rotate_bwd_kernel(RotateArgs a, int lanes,
                                                              int64_t units) {
  const int j = threadIdx.x & (lanes - 1);
  const int groups = kThreads / lanes;
  const Place p = place_of<V, INTER>(j, a.dim, a.rot);
  const float inv = 1.0f / (float)a.dim;
  float acc[2][2 * V];
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) acc[0][i] = acc[1][i] = 0.0f;
  for (int64_t unit = (int64_t)blockIdx.x * groups + threadIdx.x / lanes; unit < units;
       unit += (int64_t)gridDim.x * groups) {
    int64_t t;
    int which, h0, n;
    unit_of<U>(a, unit, t, which, h0, n);
    float x[U][2 * V], g[U][2 * V];
    const IO* in = static_cast<const IO*>(a.x[which]) + t * a.stride[which] + (int64_t)h0 * a.dim;
    const IO* dy =
        static_cast<const IO*>(a.dy[which]) + t * a.dstride[which] + (int64_t)h0 * a.dim;
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) x[u][i] = g[u][i] = 0.0f;
      if (p.on && u < n) {
        load_pairs<IO, V, INTER>(in + u * a.dim, p, x[u]);
        load_pairs<IO, V, INTER>(dy + u * a.dim, p, g[u]);
      }
    }
    float c[V], s[V], w[2 * V];
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) w[i] = 1.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = 1.0f, s[i] = 0.0f;
    if (p.on) {
      load_turn<V>(a, t, p, c, s);
      if (a.w[which]) load_pairs<float, V, INTER>(a.w[which], p, w);
    }
    IO* out = static_cast<IO*>(a.out[which]) + (t * a.heads[which] + h0) * a.dim;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float ss = 0.0f, dot = 0.0f;
      float wg[2 * V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float ga = g[u][i], gb = g[u][V + i];
        g[u][i] = ga * c[i] + gb * s[i];
        g[u][V + i] = gb * c[i] - ga * s[i];
      }
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) {
        wg[i] = w[i] * g[u][i];
        ss = __builtin_fmaf(x[u][i], x[u][i], ss);
        dot = __builtin_fmaf(wg[i], x[u][i], dot);
      }
      for (int m = 1; m < lanes; m <<= 1) {
        ss += __shfl_xor(ss, m);
        dot += __shfl_xor(dot, m);
      }
      const float r = rsqrtf(__builtin_fmaf(ss, inv, a.eps));
      const float k = dot * inv * r * r;  // mean(w g x r) * r
      float dx[2 * V];
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) {
        dx[i] = r * (wg[i] - x[u][i] * k);
        const float dw = g[u][i] * x[u][i] * r;
        acc[0][i] += which ? 0.0f : dw;
        acc[1][i] += which ? dw : 0.0f;
      }
      if (p.on && u < n) store_pairs<IO, V, INTER>(out + u * a.dim, p, dx);
    }
  }
  if (!a.dw_part) return;
  extern __shared__ float part[];  // [groups, dim]
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    float* mine = part + (threadIdx.x / lanes) * a.dim;
    if (p.on) store_pairs<float, V, INTER>(mine, p, acc[which]);
    __syncthreads();
    for (int d = threadIdx.x; d < a.dim; d += kThreads) {
      float sum = 0.0f;
      for (int i = 0; i < groups; ++i) sum += part[i * a.dim + d];
      a.dw_part[((int64_t)blockIdx.x * 2 + which) * a.dim + d] = sum;
    }
  }
}

// dw[which][d] = sum over blocks of part[block, which, d]; 16 threads to a
// channel, each a run of blocks, added in order.
__global__ __launch_bounds__(256) void rotate_dw_kernel(RotateArgs a, int blocks) {
  __shared__ float part[16][17];
  const int col = blockIdx.x * 16 + (threadIdx.x & 15), row = threadIdx.x >> 4;
  const int which = blockIdx.y;
  if (!a.dw[which]) return;
  float s = 0.0f;
  if (col < a.dim)
    for (int b = row; b < blocks; b += 16) s += a.dw_part[((int64_t)b * 2 + which) * a.dim + col];
  part[row][threadIdx.x & 15] = s;
  __syncthreads();
  if (row == 0 && col < a.dim) {
    float t = 0.0f;
    for (int i = 0; i < 16; ++i) t += part[i][threadIdx.x & 15];
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
template <int U> int64_t units_of(const RotateArgs& a) {
  return a.tokens * ((a.heads[0] + U - 1) / U + (a.heads[1] + U - 1) / U);
}

template <typename IO, int V, bool INTER>
hipError_t fwd_v(const RotateArgs& a, hipStream_t stream) {
  const int lanes = lanes_of(a.dim, V);
  constexpr int U = 2;
  const int64_t units = units_of<U>(a), per = kThreads / lanes;
  hipLaunchKernelGGL((rotate_fwd_kernel<IO, V, INTER, U>), dim3((unsigned)((units + per - 1) / per)),
                     dim3(kThreads), 0, stream, a, lanes, units);
  return hipGetLastError();
}

template <typename IO, int V, bool INTER>
hipError_t bwd_v(const RotateArgs& a, hipStream_t stream) {
  const int lanes = lanes_of(a.dim, V), groups = kThreads / lanes;
  constexpr int U = 2;
  const int blocks = rotate_bwd_blocks(a.tokens, a.heads[0] + a.heads[1], a.dim);
  hipLaunchKernelGGL((rotate_bwd_kernel<IO, V, INTER, U>), dim3(blocks), dim3(kThreads),
                     (size_t)groups * a.dim * 4, stream, a, lanes, units_of<U>(a));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dw_part) return e;
  hipLaunchKernelGGL(rotate_dw_kernel, dim3((a.dim + 15) / 16, 2), dim3(256), 0, stream, a, blocks);
  return hipGetLastError();
}

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

// Blocks of the backward: four to a CU, fewer when there are not that many
// rows.
int rotate_bwd_blocks(int64_t tokens, int heads, int dim) {
  const int64_t want = (tokens * heads * dim + 8191) / 8192;
  return (int)(want < 1 ? 1 : want > 1024 ? 1024 : want);
}

hipError_t launch_rotate_fwd(const RotateArgs& a, bool io_bf16, hipStream_t stream) {
  return launch<false>(a, io_bf16, stream);
}
hipError_t launch_rotate_bwd(const RotateArgs& a, bool io_bf16, hipStream_t stream) {
  return launch<true>(a, io_bf16, stream);
}

}  // namespace ssm
