// ssm_delta_prep.hip -- what the chunks of the gated delta rule need besides their
// tokens, for all chunks at once (gfx950, wave64).
//
// In a chunk that the state S enters, r_t = v_t - exp(G_t) S k_t - sum over s < t
// of N_ts b_s r_s, with N_ts = exp(G_t - G_s) k_t . k_s: r = (1 + N b)^-1 (v -
// exp(G) k S^T).  The inverse does not depend on the state, and neither do P_ts =
// scale exp(G_t - G_s) q_t . k_s: one wave per chunk and head forms them here and
// leaves them as the operands that the walks read (ssm_delta.h).
//
// Both inverses, (1 + N b)^-1 = 1 + M b and (1 + b N)^-1 = 1 + b M, come from one
// strictly lower M = -(1 + N b)^-1 N, which takes N's place block by block: the
// four blocks of 16 on the diagonal by substitution, a lane to a column, the ones
// below them by products of blocks, M10 = -(1 + M11 b1) N10 (1 + b0 M00), first of
// 16, then of 32.  (A series in powers of N b would need no substitution, but for
// like keys and beta near 1 the powers reach 1e18 and cancel.)
//
// The sums of the log decays are taken in 64 bits and their differences in two fp32
// parts, so that an exp is as good as its own argument, however far the sums go: of a
// difference d, rounded to fp32, off by |d| 2^-24 of itself, which is under 2^-25 of 1.
// Decays below -1e4, -inf among them, count as -1e4, whose exp is 0 in whatever sum.
#include <algorithm>

#include "ssm_delta_mm.h"

namespace ssm {
namespace {

constexpr int kLd = 20;  // a row of a 16 x 16 block in LDS: no bank twice by rows or columns

__device__ __forceinline__ void wave_sync() {  // orders a wave's accesses to its LDS
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A fragment of fp32 values: the lanes' first four, then their last four.
__device__ __forceinline__ void put_floats(uint8_t* f, int lane, const float* x) {
  *reinterpret_cast<f32x4_t*>(f + lane * 16) = f32x4_t{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4_t*>(f + 1024 + lane * 16) = f32x4_t{x[4], x[5], x[6], x[7]};
}

// A wave's LDS: the ten blocks (i, j), j <= i, of a lower triangle, and by token G
// in two parts and beta.
struct PrepShared {
  float m[10 * 16 * kLd];
  float hi[C], lo[C], b[C];
  __device__ __forceinline__ static int at(int t, int s) {  // of entry (t, s)
    const int i = t >> 4, j = s >> 4;
    return ((i * (i + 1) / 2 + j) * 16 + (t & 15)) * kLd + (s & 15);
  }
};

// N, whose entries below the diagonal stand in sh.m (zeros on and above it in the
// blocks of the diagonal), becomes M.
__device__ __forceinline__ void solve(PrepShared& sh, int lane) {
  const int r16 = lane & 15, g = lane >> 4;
  float* m = sh.m;
  {
    float* a = m + PrepShared::at(16 * g, 16 * g);  // a block to each lane group
    float x[16], bx[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float sum = a[i * kLd + r16];
#pragma unroll
      for (int l4 = 0; l4 < i; l4 += 4) {
        const f32x4_t row = *reinterpret_cast<const f32x4_t*>(a + i * kLd + l4);
#pragma unroll
        for (int l = 0; l < 4; ++l)
          if (l4 + l < i) sum = __builtin_fmaf(row[l], bx[l4 + l], sum);
      }
      x[i] = i > r16 ? -sum : 0.0f;
      bx[i] = sh.b[16 * g + i] * x[i];
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i * kLd + r16] = x[i];
    wave_sync();
  }
  // products of blocks: left operands by rows, right ones by columns; a result is a
  // right operand as it stands
  auto left = [&](int i, int j) {
    return *reinterpret_cast<const f32x4_t*>(m + PrepShared::at(16 * i + r16, 16 * j + 4 * g));
  };
  auto right = [&](int i, int j) {
    f32x4_t v;
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = m[PrepShared::at(16 * i + 4 * g + x, 16 * j + r16)];
    return v;
  };
  f32x4_t b[4], unit;  // betas of the tokens 4 g .. of a block; the diagonal
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const f32x4_t*>(sh.b + 16 * i + 4 * g);
#pragma unroll
  for (int x = 0; x < 4; ++x) unit[x] = 4 * g + x == r16 ? 1.0f : 0.0f;
  auto mm = [&](f32x4_t a, f32x4_t v, f32x4_t c) {
#pragma unroll
    for (int x = 0; x < 4; ++x) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[x], v[x], c, 0, 0, 0);
    return c;
  };
  auto put = [&](int i, int j, f32x4_t v) {
#pragma unroll
    for (int x = 0; x < 4; ++x) m[PrepShared::at(16 * i + 4 * g + x, 16 * j + r16)] = v[x];
  };
  const f32x4_t none{0, 0, 0, 0};
  {
    const f32x4_t z1 = mm(left(1, 0), right(0, 0) * b[0] + unit, none);
    const f32x4_t z3 = mm(left(3, 2), right(2, 2) * b[2] + unit, none);
    const f32x4_t t1 = -mm(left(1, 1) * b[1] + unit, z1, none);
    const f32x4_t t3 = -mm(left(3, 3) * b[3] + unit, z3, none);
    wave_sync();
    put(1, 0, t1);
    put(3, 2, t3);
    wave_sync();
  }
  f32x4_t z[2][2];
  {
    const f32x4_t t00 = right(0, 0) * b[0] + unit, t10 = right(1, 0) * b[1],
                  t11 = right(1, 1) * b[1] + unit;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4_t n0 = left(2 + i, 0), n1 = left(2 + i, 1);
      z[i][0] = mm(n1, t10, mm(n0, t00, none));
      z[i][1] = mm(n1, t11, none);
    }
  }
  const f32x4_t t22 = left(2, 2) * b[2] + unit, t32 = left(3, 2) * b[2],
                t33 = left(3, 3) * b[3] + unit;
  wave_sync();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    put(2, j, -mm(t22, z[0][j], none));
    put(3, j, -mm(t33, z[1][j], mm(t32, z[0][j], none)));
  }
  wave_sync();
}

// Of the products of the chunk's keys and queries a lane holds column r16 of a tile
// and rows 4 g + x, both in the interleaved order of ssm_delta_mm.h.  Forward the
// rows are the tokens s, which two tiles make the slots of P's right operand, and
// the columns t; BACK the other way round.
template <typename IO, int KD, bool BACK>
__global__ __launch_bounds__(256, 2) void delta_prep_kernel(DeltaArgs a, int64_t block0) {
  typedef Mat<IO> M;
  constexpr int KS = KD / 32;
  constexpr DeltaRecord R = delta_record(BACK);
  __shared__ PrepShared waves[4];
  PrepShared& sh = waves[wave_id()];
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  const int64_t id = (block0 + blockIdx.x) * 4 + wave_id();
  const int64_t chunk = id / a.heads;
  const int head = (int)(id - chunk * a.heads);
  if (chunk >= (a.cu ? (int64_t)a.table[a.nseq] : a.chunks)) return;
  const Chunk c = chunk_of(a, chunk);
  uint8_t* rec = a.record + id * R.size;
  float* rows = reinterpret_cast<float*>(rec + R.rows);

  // rows of the keys and queries: of token t, 8 channels from 32 ks + 8 g on
  const uint32_t k_row = (uint32_t)a.k.stride * (uint32_t)sizeof(IO),
                 q_row = (uint32_t)a.q.stride * (uint32_t)sizeof(IO);
  auto resource = [&](const DeltaOperand& o, uint32_t row) {
    return make_rsrc(static_cast<const IO*>(o.p) + c.t0 * o.stride + (int64_t)(head / o.hdiv) * a.kd,
                     (uint32_t)(c.n - 1) * row + (uint32_t)a.kd * (uint32_t)sizeof(IO));
  };
  const __amdgpu_buffer_rsrc_t rk = resource(a.k, k_row), rq = resource(a.q, q_row);
  auto load_row = [&](__amdgpu_buffer_rsrc_t r, uint32_t row, int t, typename M::In* to) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int col = 32 * ks + 8 * g;
      const uint32_t at = col < a.kd ? (uint32_t)t * row + (uint32_t)col * (uint32_t)sizeof(IO)
                                     : 0x7f000000u;
      if constexpr (sizeof(IO) == 2) {
        to[ks] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
      } else {
        to[ks].lo = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
        to[ks].hi =
            __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16, 0, 0));
      }
    }
  };
  float ld = 0.0f, beta = 0.0f;
  if (lane < c.n) {
    const int64_t at = (c.t0 + lane) * a.heads + head;
    ld = a.log_decay[at];
    beta = io<IO>::load(static_cast<const IO*>(a.beta) + at);
  }
  // (Memory answers in order, stores among the loads: the rows of q are asked for
  // before the first store.  With that, and with two blocks a CU in place of three,
  // which spilled, a backward's 10240 heads of 128 by chunks take 111 us in place of
  // 145, 6144 of 64 64 in place of 78.)
  constexpr bool AHEAD = sizeof(IO) == 2;  // (fp32: no registers for it)
  constexpr int kHeld = AHEAD ? 4 : 1;
  typename M::In k[4][KS], qs[kHeld][KS];
#pragma unroll
  for (int tt = 0; tt < 4; ++tt) load_row(rk, k_row, row_of(tt, r16), k[tt]);
#pragma unroll
  for (int tt = 0; tt < (AHEAD ? 4 : 0); ++tt) load_row(rq, q_row, row_of(tt, r16), qs[tt]);

  // decays and betas: lane l is token l
  double G_end;
  float lam, gam, odd = beta * 0.0f + (ld < 0.0f ? 0.0f : ld * 0.0f);  // NaN where one is not finite
  {
    double G = (double)(ld < -1e4f ? -1e4f : ld) * 1.4426950408889634;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double up = __shfl_up(G, d);
      if (lane >= d) G += up;
    }
    G_end = __shfl(G, 63);
    const float hi = (float)G, lo = (float)(G - (double)hi);
    sh.hi[lane] = hi;
    sh.lo[lane] = lo;
    sh.b[lane] = beta;
    lam = fast_exp2(hi) * (1.0f + 0.6931471806f * lo);
    gam = fast_exp2((float)(G_end - G));
  }
  wave_sync();

  // N by entries into LDS, P as fragments into the record: the pair's tiles (2 p,
  // 2 p + 1) of rows against a tile of columns
#pragma unroll
  for (int tt = 0; tt < 4; ++tt) {
    const int here = row_of(tt, r16);  // the column's token
    const float hi = sh.hi[here], lo = sh.lo[here];
    if (!AHEAD && !BACK) load_row(rq, q_row, here, qs[0]);
#pragma unroll
    for (int ks = BACK ? tt >> 1 : 0; ks < (BACK ? 2 : (tt >> 1) + 1); ++ks) {
      float pairs[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int rt = 2 * ks + half;
        if (!AHEAD && BACK) load_row(rq, q_row, row_of(rt, r16), qs[0]);
        const typename M::In(&q)[KS] = qs[!AHEAD ? 0 : BACK ? rt : tt];
        f32x4_t n{0, 0, 0, 0}, p{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
          for (int i = 0; i < M::steps((typename M::In*)nullptr, (typename M::In*)nullptr); ++i) {
            n = M::step(k[rt][kk], k[tt][kk], n, i);
            p = BACK ? M::step(q[kk], k[tt][kk], p, i) : M::step(k[rt][kk], q[kk], p, i);
          }
        }
        const int first = 32 * ks + 8 * g + 4 * half;  // the tokens of the rows, from this on
        const f32x4_t oh = *reinterpret_cast<const f32x4_t*>(sh.hi + first);
        const f32x4_t ol = *reinterpret_cast<const f32x4_t*>(sh.lo + first);
        const f32x4_t ob = *reinterpret_cast<const f32x4_t*>(sh.b + first);
        f32x4_t e;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int other = first + x;
          const float d = (hi - oh[x]) + (lo - ol[x]), w = fast_exp2(BACK ? -d : d);
          // (selects: beyond the diagonal w may be infinite)
          const float v = p[x] * w * a.scale;
          pairs[4 * half + x] = (BACK ? here <= other : other <= here) ? (BACK ? v : v * ob[x]) : 0.0f;
          e[x] = (BACK ? here < other : other < here) ? n[x] * w : 0.0f;
          odd = __builtin_fmaf(e[x], 0.0f, odd);
        }
        if (BACK) {
          if ((here >> 4) <= (first >> 4)) {
            float* to = sh.m + PrepShared::at(first, here);
#pragma unroll
            for (int x = 0; x < 4; ++x) to[x * kLd] = e[x];
          }
        } else if ((first >> 4) <= (here >> 4)) {
          *reinterpret_cast<f32x4_t*>(sh.m + PrepShared::at(here, first)) = e;
        }
      }
      uint8_t* to = rec + R.pairs + frag_of<BACK>(tt, ks) * kDeltaFragBytes;
      if constexpr (BACK || sizeof(IO) == 4)
        put_floats(to, lane, pairs);
      else
        M::template put<2>(to, lane, M::template split<2>(pairs));
    }
  }
  rows[kRowLam * C + lane] = lam;
  rows[kRowGam * C + lane] = gam;
  rows[kRowBeta * C + lane] = beta;
  rows[kRowDecay * C + lane] = fast_exp2(ld * kLog2e);
  rows[kRowG * C + lane] = sh.hi[lane];
  rows[kRowGLow * C + lane] = sh.lo[lane];
  const bool any = __ballot(!(odd == 0.0f)) != 0;
  if (lane < 3) {
    const double all = exp2(G_end);
    const float near = (float)all, low = fabsf(near) <= 3.4028235e38f ? (float)(all - (double)near) : 0.0f;
    rows[kDeltaRows * C + lane] = lane == 0 ? near : lane == 1 ? low : any ? 1.0f : 0.0f;
  }
  wave_sync();
  solve(sh, lane);

  // 1 + M b by rows
#pragma unroll
  for (int f = 0; f < kDeltaFrags; ++f) {
    const FragAt fa = frag_at<false>(f);
    const int t = row_of(fa.tt, r16), s0 = 32 * fa.ks + 8 * g;
    float x[8];
    const bool on = (s0 >> 4) <= (t >> 4);
    const float* from = sh.m + (on ? PrepShared::at(t, s0) : 0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_t m = *reinterpret_cast<const f32x4_t*>(from + 4 * h);
      const f32x4_t b = *reinterpret_cast<const f32x4_t*>(sh.b + s0 + 4 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = s0 + 4 * h + j;
        x[4 * h + j] = s < t ? m[j] * b[j] : s == t ? 1.0f : 0.0f;
      }
    }
    put_floats(rec + R.solve + f * kDeltaFragBytes, lane, x);
  }
  if constexpr (BACK) {  // (1 + b M)^T by rows
#pragma unroll
    for (int f = 0; f < kDeltaFrags; ++f) {
      const FragAt fa = frag_at<true>(f);
      const int s = row_of(fa.tt, r16), u0 = 32 * fa.ks + 8 * g;
      float x[8];
      const bool on = (s >> 4) <= (u0 >> 4);
      const float* from = sh.m + (on ? PrepShared::at(u0, s) : 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = u0 + j;
        x[j] = s < t ? from[j * kLd] * sh.b[t] : s == t ? 1.0f : 0.0f;
      }
      put_floats(rec + R.back + f * kDeltaFragBytes, lane, x);
    }
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
  // the sum of the strip's numbers before this thread's; `all` of them
  auto before = [&](long long n, long long& all) {
    long long sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const long long v = __shfl_up(sum, d);
      if ((i & 63) >= d) sum += v;
    }
    if ((i & 63) == 63) upto[i >> 6] = sum;
    __syncthreads();
    all = 0;
    for (int w = 0; w < kStrip / 64; ++w) {
      if (w < (i >> 6)) sum += upto[w];
      all += upto[w];
    }
    __syncthreads();
    return sum - n;
  };
  int32_t* spans = a.table + 2 * a.nseq + 1;
  long long base = 0, span_base = 0;
  for (int64_t s0 = 0; s0 < a.nseq; s0 += kStrip) {
    const int64_t seq = s0 + i;
    long long n = 0, all;
    if (seq < a.nseq) {
      const int first = clamp_token(a.cu[seq], (int)a.tokens);
      const int end = clamp_token(a.cu[seq + 1], (int)a.tokens);
      n = end > first ? ((int64_t)end - first + C - 1) / C : 0;
      if (seq < kRanked) count[seq] = (int)n;
    }
    const long long from = base + before(n, all), most = a.chunks;
    if (seq < a.nseq) a.table[seq] = (int)min(from, most);
    base += all;
    if (a.span_chunks > 0) {  // (of the chunks that there is room for; one at least)
      const long long held = min(from + n, most) - min(from, most);
      n = seq < a.nseq ? max((held + a.span_chunks - 1) / a.span_chunks, 1ll) : 0;
      const long long at = span_base + before(n, all);
      if (seq < a.nseq) spans[seq] = (int)at;
      span_base += all;
    }
  }
  if (i == 0 && a.span_chunks > 0) spans[a.nseq] = (int)span_base;
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

template <typename IO, int KD, bool BACK>
hipError_t launch(const DeltaArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.chunks * a.heads + 3) / 4;
  for (int64_t b = 0; b < blocks; b += max_blocks(256)) {
    const dim3 grid((unsigned)std::min<int64_t>(blocks - b, max_blocks(256)));
    hipLaunchKernelGGL((delta_prep_kernel<IO, KD, BACK>), grid, dim3(256), 0, stream, a, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <typename IO, int KD> hipError_t launch_kd(const DeltaArgs& a, hipStream_t stream) {
  return a.back ? launch<IO, KD, true>(a, stream) : launch<IO, KD, false>(a, stream);
}

}  // namespace

hipError_t launch_delta_table(const DeltaArgs& a, hipStream_t stream) {
  if (!a.cu) return hipSuccess;
  hipLaunchKernelGGL(delta_table_kernel, dim3(1), dim3(kStrip), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_delta_prep(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  if (a.kd <= 64) return io_bf16 ? launch_kd<bf16, 64>(a, stream) : launch_kd<float, 64>(a, stream);
  return io_bf16 ? launch_kd<bf16, 128>(a, stream) : launch_kd<float, 128>(a, stream);
}

}  // namespace ssm
