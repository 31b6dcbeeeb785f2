// ssm_delta_prep.hip -- what the chunks of the gated delta rule need besides their
// tokens, for all chunks at once (gfx950, wave64).
//
// In a chunk that the state S enters, r_t = v_t - exp(G_t) S k_t - sum over s < t
// of N_ts b_s r_s, with N_ts = exp(G_t - G_s) k_t . k_s: r = (1 + N b)^-1 (v -
// exp(G) k S^T).  The inverse does not depend on the state, so one wave per chunk
// and head writes it here: the 64 x 64 product of the keys on the matrix cores,
// the decays between its tokens, and the inverse of the unit lower triangle by
// blocks: the four of 16 by substitution, a lane to a column, the ones below them
// by products of blocks, T10 = -T11 A10 T00, first of 16, then of 32.  (A series
// in powers of the triangle would need no substitution, but for like keys and
// beta near 1 the powers reach 1e18 and cancel.)
//
// The sums of the log decays are taken in 64 bits, so that exp of a difference is
// good to fp32 however far the sums go; decays below -1e4, -inf among them, count
// as -1e4, whose exp is 0 in whatever sum.
#include <algorithm>

#include "ssm_delta_mm.h"

namespace ssm {
namespace {

constexpr int kLd = C + 4;  // a row of the triangle in LDS

__device__ __forceinline__ void wave_sync() {  // orders a wave's accesses to its LDS
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ double shfl_up(double v, int d) { return __shfl_up(v, d); }

// The inverse of the unit lower triangle whose entries below the diagonal stand in
// m, in its place, zeros above the diagonal.
__device__ __forceinline__ void invert(float* m, int lane) {
  const int r16 = lane & 15, g = lane >> 4;
  {
    const float* a = m + (16 * g) * kLd + 16 * g;  // a block of 16 to each lane group
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = i == r16 ? 1.0f : 0.0f;
#pragma unroll
      for (int l4 = 0; l4 < i; l4 += 4) {
        const f32x4_t row = *reinterpret_cast<const f32x4_t*>(a + i * kLd + l4);
#pragma unroll
        for (int l = 0; l < 4; ++l)
          if (l4 + l < i) x[i] = __builtin_fmaf(-row[l], x[l4 + l], x[i]);
      }
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 16; ++i) m[(16 * g + i) * kLd + 16 * g + r16] = x[i];
    wave_sync();
  }
  // products of blocks: left operands by rows, right ones by columns; a result is
  // a right operand as it stands
  auto left = [&](int i, int j) {
    return *reinterpret_cast<const f32x4_t*>(m + (16 * i + r16) * kLd + 16 * j + 4 * g);
  };
  auto right = [&](int i, int j) {
    f32x4_t v;
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = m[(16 * i + 4 * g + x) * kLd + 16 * j + r16];
    return v;
  };
  auto mm = [&](f32x4_t a, f32x4_t b, f32x4_t c) {
#pragma unroll
    for (int x = 0; x < 4; ++x) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[x], b[x], c, 0, 0, 0);
    return c;
  };
  auto put = [&](int i, int j, f32x4_t v) {
#pragma unroll
    for (int x = 0; x < 4; ++x) m[(16 * i + 4 * g + x) * kLd + 16 * j + r16] = v[x];
  };
  const f32x4_t none{0, 0, 0, 0};
  {
    const f32x4_t z1 = mm(left(1, 0), right(0, 0), none), z3 = mm(left(3, 2), right(2, 2), none);
    const f32x4_t t1 = -mm(left(1, 1), z1, none), t3 = -mm(left(3, 3), z3, none);
    wave_sync();
    put(1, 0, t1);
    put(3, 2, t3);
    put(0, 1, none);
    put(2, 3, none);
    wave_sync();
  }
  f32x4_t z[2][2], t[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    z[i][0] = mm(left(2 + i, 1), right(1, 0), mm(left(2 + i, 0), right(0, 0), none));
    z[i][1] = mm(left(2 + i, 1), right(1, 1), none);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    t[0][j] = -mm(left(2, 2), z[0][j], none);
    t[1][j] = -mm(left(3, 3), z[1][j], mm(left(3, 2), z[0][j], none));
  }
  wave_sync();
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) put(2 + i, j, t[i][j]);
  wave_sync();
}

template <typename IO, int KD>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, int64_t block0) {
  typedef Mat<IO> M;
  constexpr int KS = KD / 32;
  struct Wave {
    float m[C * kLd];
    double g[C];
    float b[C];
  };
  __shared__ Wave waves[4];
  Wave& sh = waves[wave_id()];
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  const int64_t id = (block0 + blockIdx.x) * 4 + wave_id();
  const int64_t chunk = id / a.heads;
  const int head = (int)(id - chunk * a.heads);
  int seq;
  if (a.cu) {
    if (chunk >= a.table[a.nseq]) return;
    int lo = 0, hi = (int)a.nseq;  // the last sequence that begins at or before the chunk
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (a.table[mid] <= chunk) lo = mid;
      else hi = mid;
    }
    seq = lo;
  } else {
    if (chunk >= a.chunks) return;
    seq = (int)(chunk / a.per);
  }
  const Seq s = seq_of(a, seq);
  const int c0 = (int)(chunk - s.chunk0) * C, n = min(s.len - c0, C);
  const int64_t t0 = s.first + c0;
  float* rec = a.record + id * delta_record(a.back);
  float* rows = rec + (a.back ? 2 : 1) * kDeltaFrags * kDeltaFrag;

  // decays and betas: lane l is token l
  float ld = 0.0f, beta = 0.0f;
  if (lane < n) {
    const int64_t at = (t0 + lane) * a.heads + head;
    ld = a.log_decay[at];
    beta = io<IO>::load(static_cast<const IO*>(a.beta) + at);
  }
  const bool odd_gate = !(fabsf(beta) <= 3.4028235e38f) || !(ld <= 3.4028235e38f);
  double G = (double)(ld < -1e4f ? -1e4f : ld) * 1.4426950408889634;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double up = shfl_up(G, d);
    if (lane >= d) G += up;
  }
  const double end = __shfl(G, 63);
  sh.g[lane] = G;
  sh.b[lane] = beta;
  rows[kRowLam * C + lane] = fast_exp2((float)G);
  rows[kRowGam * C + lane] = fast_exp2((float)(end - G));
  rows[kRowBeta * C + lane] = beta;
  rows[kRowDecay * C + lane] = fast_exp2(ld * kLog2e);
  rows[kRowG * C + lane] = (float)G;
  rows[kRowGLow * C + lane] = (float)(G - (double)(float)G);

  // the keys' products
  typename M::In k[4][KS];
  const IO* kp = static_cast<const IO*>(a.k.p) + t0 * a.k.stride + (int64_t)(head / a.k.hdiv) * a.kd;
  bool odd = odd_gate;
#pragma unroll
  for (int tt = 0; tt < 4; ++tt) {
    const int t = 16 * tt + r16;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int c = 32 * ks + 8 * g;
      k[tt][ks] = M::zero();
      if (t < n && c < a.kd)
        k[tt][ks] = *reinterpret_cast<const typename M::In*>(kp + (int64_t)t * a.k.stride + c);
      odd |= M::odd(k[tt][ks]);
    }
  }
  wave_sync();
  f32x4_t N[4][4];  // [i][j], j <= i: rows t = 16 i + 4 g + x, column s = 16 j + r16
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double gs = sh.g[16 * j + r16];
#pragma unroll
    for (int i = j; i < 4; ++i) {
      f32x4_t m{0, 0, 0, 0};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) m = M::mm(k[i][ks], k[j][ks], m);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int t = 16 * i + 4 * g + x;
        const float w = fast_exp2((float)(sh.g[t] - gs));
        N[i][j][x] = t > 16 * j + r16 ? w * m[x] : 0.0f;
        odd |= !(fabsf(N[i][j][x]) <= 3.4028235e38f);
      }
    }
  }

#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (side == 1 && !a.back) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float bs = sh.b[16 * j + r16];
#pragma unroll
      for (int i = j; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int t = 16 * i + 4 * g + x;
          sh.m[t * kLd + 16 * j + r16] = N[i][j][x] * (side ? sh.b[t] : bs);
        }
    }
    wave_sync();
    invert(sh.m, lane);
    float* out = rec + side * kDeltaFrags * kDeltaFrag + lane * 8;
#pragma unroll
    for (int f = 0; f < kDeltaFrags; ++f) {
      f32x4_t lo, hi;
      if (side == 0) {  // rows t of tile tt, columns s: (0..3, 0), (2, 1), (3, 1)
        const int tt = f < 4 ? f : f - 2, ks = f < 4 ? 0 : 1;
        const float* p = sh.m + row_of(tt, r16) * kLd + 32 * ks + 8 * g;
        lo = *reinterpret_cast<const f32x4_t*>(p);
        hi = *reinterpret_cast<const f32x4_t*>(p + 4);
      } else {  // rows s of tile tt, columns t: (0, 0), (0, 1), (1, 0), (1, 1), (2, 1), (3, 1)
        const int tt = f < 4 ? f >> 1 : f - 2, ks = f < 4 ? f & 1 : 1;
        const float* p = sh.m + (32 * ks + 8 * g) * kLd + row_of(tt, r16);
#pragma unroll
        for (int j = 0; j < 4; ++j) lo[j] = p[j * kLd], hi[j] = p[(4 + j) * kLd];
      }
      *reinterpret_cast<f32x4_t*>(out + f * kDeltaFrag) = lo;
      *reinterpret_cast<f32x4_t*>(out + f * kDeltaFrag + 4) = hi;
    }
    wave_sync();
  }
  const bool any = __ballot(odd) != 0;
  if (lane < 3) {
    const double all = exp2(end);
    const float near = (float)all;
    const float rest = near <= 3.4028235e38f ? (float)(all - (double)near) : 0.0f;
    rows[kDeltaRows * C + lane] = lane == 0 ? near : lane == 1 ? rest : (any ? 1.0f : 0.0f);
  }
}

// Packed sequences: the first chunk of each (and of none), and the sequences from
// the one with most chunks to the one with least, so that the walks that take
// longest start first: one block, in strips; ranks are counted, up to kRanked
// sequences (so many walks even out by themselves).  Sums are 64-bit: cu_seqlens
// that run up and down make sequences that overlap, and more chunks than the
// workspace holds; those past its end are left out.
constexpr int kStrip = 1024, kRanked = 4096;
__global__ __launch_bounds__(kStrip) void delta_table_kernel(DeltaArgs a) {
  __shared__ long long upto[kStrip / 64];
  __shared__ int count[kRanked];
  const int i = threadIdx.x;
  long long base = 0;
  for (int64_t s0 = 0; s0 < a.nseq; s0 += kStrip) {
    const int64_t seq = s0 + i;
    long long n = 0;
    if (seq < a.nseq) {
      const int first = clamp_token(a.cu[seq], (int)a.tokens);
      const int end = clamp_token(a.cu[seq + 1], (int)a.tokens);
      n = end > first ? ((int64_t)end - first + C - 1) / C : 0;
      if (seq < kRanked) count[seq] = (int)n;
    }
    long long sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const long long v = __shfl_up(sum, d);
      if ((i & 63) >= d) sum += v;
    }
    if ((i & 63) == 63) upto[i >> 6] = sum;
    __syncthreads();
    long long all = 0;
    for (int w = 0; w < kStrip / 64; ++w) {
      if (w < (i >> 6)) sum += upto[w];
      all += upto[w];
    }
    if (seq < a.nseq) a.table[seq] = (int)min(base + sum - n, (long long)a.chunks);
    base += all;
    __syncthreads();
  }
  if (i == 0) a.table[a.nseq] = (int)min(base, (long long)a.chunks);
  int* order = a.table + a.nseq + 1;
  for (int64_t seq = i; seq < a.nseq; seq += kStrip) {
    int64_t rank = seq;
    if (a.nseq <= kRanked) {
      const int mine = count[seq];
      rank = 0;
      for (int o = 0; o < (int)a.nseq; ++o)
        rank += count[o] > mine || (count[o] == mine && o < (int)seq);
    }
    order[rank] = (int)seq;
  }
}

template <typename IO, int KD> hipError_t launch(const DeltaArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.chunks * a.heads + 3) / 4;
  for (int64_t b = 0; b < blocks; b += max_blocks(256)) {
    const dim3 grid((unsigned)std::min<int64_t>(blocks - b, max_blocks(256)));
    hipLaunchKernelGGL((delta_prep_kernel<IO, KD>), grid, dim3(256), 0, stream, a, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_delta_table(const DeltaArgs& a, hipStream_t stream) {
  if (!a.cu) return hipSuccess;
  hipLaunchKernelGGL(delta_table_kernel, dim3(1), dim3(kStrip), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_delta_prep(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  if (a.kd <= 64) return io_bf16 ? launch<bf16, 64>(a, stream) : launch<float, 64>(a, stream);
  return io_bf16 ? launch<bf16, 128>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace ssm
