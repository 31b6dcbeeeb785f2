// ssm_linattn_walk.h -- what the chunked walks of the linear attention share
// (ssm_linattn_mm.hip, ssm_linattn_f32.hip): decays, units of work, block
// numbering.
#pragma once

#include "ssm_device.h"
#include "ssm_linattn.h"

namespace ssm {

// Up to four walks of the same head sizes in one launch (the backward's): the
// walks of a head side by side, so that those that read the same tiles share an
// L2.
struct LinWalks {
  LinArgs a[4];
  int n;
};

// Replaces the end states of the segments (the first one's, the others' own) by
// the states entering them (with dg_part, the state's derivative too).
hipError_t launch_lin_carry(const LinWalks& ws, hipStream_t stream);

namespace {

// log2 of the decay, finite when it is -inf, so that power(., 0) is 1 then too
// (and power(., n) 0 for n > 0).
__device__ __forceinline__ float log2_decay(float log_decay) {
  const float g2 = log_decay * kLog2e;
  return g2 < -3e38f ? -3e38f : g2;
}
// a^n for n >= 0.
__device__ __forceinline__ float power(float g2, int n) { return fast_exp2(g2 * (float)n); }

// a^n again and again, for a state that takes in many pieces of n tokens: the
// number next to a^n, or its neighbour on the other side of it in the share that
// makes their product, of however many, that power but for a rounding.  One
// factor off by the same half unit every time would bring 65536 tokens, 64 at a
// time, 3e-5 away from a decay near 1.
struct Decays {
  float near, next, share;
};
__device__ __forceinline__ Decays decays(float log_decay, int n) {
  const double e = exp2((double)log_decay * 1.4426950408889634 * n);
  Decays d{(float)e, (float)e, 0.0f};
  if (e > 1e-30 && e < 3e38) {  // (else it is 0, infinite or NaN, or leaves nothing)
    const double rest = e - (double)d.near;
    d.next = __uint_as_float(__float_as_uint(d.near) + (rest > 0.0 ? 1u : ~0u));
    d.share = (float)(rest / ((double)d.next - (double)d.near));
  }
  return d;
}
// The i-th factor: the neighbour where the sum of shares passes a half.
__device__ __forceinline__ float decay_of(const Decays& d, int i) {
  const float at = __builtin_floorf(__builtin_fmaf((float)i, d.share, 0.5f));
  return __builtin_floorf(__builtin_fmaf((float)(i + 1), d.share, 0.5f)) > at ? d.next : d.near;
}
// In scalar registers, for a decay that is the whole wave's.
__device__ __forceinline__ float scalar(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}
__device__ __forceinline__ Decays wave_decays(float log_decay, int n) {
  const Decays d = decays(log_decay, n);
  return {scalar(d.near), scalar(d.next), scalar(d.share)};
}

// Block barrier that orders LDS only: loads of the next chunk and stores of
// results stay in flight over it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A unit's tokens: p0 .. p0 + n - 1 of its sequence in walk order.  Token
// numbers fit 32 bits, and so does the end of the last chunk (at most 2^31 - 64
// tokens).
struct Unit {
  int seq, first, len;  // sequence, its first token and its length
  int seg, p0, n;
  int seg_len;          // of the sequence's segments past the first (0: uncut)
};

__device__ __forceinline__ int clamp_token(int t, int tokens) {
  return t < 0 ? 0 : t > tokens ? tokens : t;
}

__device__ __forceinline__ void sequence_of(const LinArgs& a, int seq, int& first, int& len) {
  if (!a.cu) {
    first = seq * (int)a.seqlen;
    len = (int)a.seqlen;
    return;
  }
  first = clamp_token(a.cu[seq], (int)a.tokens);
  const int end = clamp_token(a.cu[seq + 1], (int)a.tokens);
  len = end > first ? end - first : 0;
}

// Tokens of a sequence's segments past the first: all of one length, or whole
// chunks that make `each` of it.
__device__ __forceinline__ int segment_len(const LinArgs& a, int len) {
  if (!a.each) return (int)a.seg_len;
  const int chunks = len > 0 ? (len - 1) / kLinChunk + 1 : 1;
  return ((chunks - 1) / a.each + 1) * kLinChunk;
}

// The u-th unit; false past the last one.
__device__ __forceinline__ bool unit_of(const LinArgs& a, uint32_t u, Unit& x) {
  x.seg = 0;
  if (a.cu) {
    if (u >= (uint32_t)a.unit_table[0]) return false;
    x.seq = a.unit_table[1 + 2 * (int64_t)u];
    x.seg = a.unit_table[2 + 2 * (int64_t)u];
  } else if (a.seg_len == 0) {
    x.seq = (int)u;
  } else {
    x.seq = (int)(u / (uint32_t)a.segs);
    x.seg = (int)u - x.seq * (int)a.segs;
  }
  sequence_of(a, x.seq, x.first, x.len);
  x.seg_len = segment_len(a, x.len);
  const int first = a.each ? x.seg_len : (int)a.first_len;
  x.p0 = x.seg == 0 ? 0 : first + (x.seg - 1) * x.seg_len;
  x.n = x.len - x.p0;
  if (a.seg_len) x.n = min(x.n, x.seg == 0 ? first : x.seg_len);
  return true;
}

// Segments of a sequence (one when it is empty or uncut).
__device__ __forceinline__ int segments_of(const LinArgs& a, int len) {
  const int seg = segment_len(a, len), first = a.each ? seg : (int)a.first_len;
  if (a.seg_len == 0 || len <= first) return 1;
  return 1 + (len - first - 1) / seg + 1;
}

// Where the sequences are cut, a first launch gathers the states of all segments
// but the last and a second walks them all; or (lead) the first walks the first
// segments, with outputs, and the second the others.  Sequences of one length:
// places of either launch, all first segments first, none that it would leave
// out.  Packed: every unit in both.
enum Pass { kWalk, kState, kLead };
struct Places {
  uint32_t first, count;
};
__device__ __forceinline__ uint32_t unit_at(const LinArgs& a, uint32_t place) {
  if (a.cu || a.seg_len == 0) return place;
  const uint32_t n = (uint32_t)a.nseq, seg = place / n;
  return (place - seg * n) * (uint32_t)a.segs + seg;
}
inline Places places_of(const LinArgs& a, Pass pass) {
  if (a.cu || a.seg_len == 0) return {0, (uint32_t)a.units};
  const uint32_t n = (uint32_t)(a.nseq * (a.segs - 1)), one = (uint32_t)a.nseq;
  return pass != kWalk ? Places{0, n} : a.lead ? Places{one, n} : Places{0, n + one};
}

// The part of `all` from place `done` on that one launch takes: blocks of `per`
// to a place (at most 2^21, by the limits on heads and strides), and `spare` that
// round its grid up.
inline Places slice_of(Places all, uint32_t done, uint32_t threads, uint32_t per, uint32_t spare) {
  const uint32_t most = (max_blocks(threads) - spare) / per, left = all.count - done;
  return {all.first + done, left < most ? left : most};
}

// Logical block number in a grid handed out round robin to the 8 XCDs: runs of
// `group` blocks, which read the same keys and values, go to one XCD and share
// its L2, and consecutive runs go to different ones.
constexpr uint32_t kMaxGroup = 4096;  // (far more than an XCD runs at once)
__device__ __forceinline__ uint32_t xcd_block(uint32_t b, uint32_t group) {
  const uint32_t round = b / (8 * group), i = b - round * 8 * group;
  return round * 8 * group + (i & 7) * group + (i >> 3);
}

}  // namespace
}  // namespace ssm
