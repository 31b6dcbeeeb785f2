// ssm_delta.h -- internal interface between the C ABI (ssm_delta_abi.cpp) and the
// kernels of the gated delta rule (ssm_delta*.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

// One token-major operand [tokens, heads / hdiv, dim]: element (t, h, d) is at
// t * stride + (h / hdiv) * dim + d.
struct DeltaOperand {
  const void* p;
  int64_t stride;  // elements between tokens
  int hdiv;        // value heads per head of this operand
};

// Sequences are cut into chunks of 64 tokens.  What a chunk of one head needs
// besides q, k and v is computed beforehand, for all chunks at once
// (ssm_delta_prep.hip), and stands in a record:
//   solve   6 fragments of the lower triangle of (1 + N b)^-1
//   pairs   6 fragments of P b; with a backward after it, of P's transpose, and
//   back    6 fragments of the upper triangle of (1 + b N)^-T
//   rows    [kDeltaRows][64] floats by token, see DeltaRow
//   ends    decay of the whole chunk, what the fp32 number leaves of it, and
//           whether the chunk has to be walked token by token
// where N_ts = exp(G_t - G_s) k_t . k_s for s < t and P_ts = scale exp(G_t - G_s)
// q_t . k_s for s <= t, G the sum of the log decays.  A fragment is an operand of a
// product as the lanes of a wave hold it (ssm_delta_mm.h), 8 fp32 values to a lane
// (P b for bf16 inputs: in two bf16 parts).  Those of a lower triangle are (row
// tile, 32 columns) (0..3, first), (2, second), (3, second), of an upper one (0,
// both), (1, both), (2, second), (3, second).
constexpr int kDeltaChunk = 64;
constexpr int kDeltaFrags = 6;
constexpr int kDeltaFragBytes = 64 * 8 * 4;
enum DeltaRow {
  kRowLam,    // exp(G_t)
  kRowGam,    // exp(G_end - G_t)
  kRowBeta,
  kRowDecay,  // exp(log_decay)
  kRowG,      // G_t log2(e), and
  kRowGLow,   // what the fp32 number leaves of it
  kDeltaRows
};
constexpr int kDeltaEnds = 64;
struct DeltaRecord {  // byte offsets
  int solve, pairs, back, rows, size;
};
constexpr DeltaRecord delta_record(bool back) {
  const int six = kDeltaFrags * kDeltaFragBytes, rows = (back ? 3 : 2) * six;
  return {0, six, 2 * six, rows, rows + (kDeltaRows * kDeltaChunk + kDeltaEnds) * 4};
}

// What a span makes of a state: S -> S X + dec S, X [kd, kd] and behind it dec and what
// its fp32 number leaves of it; in whole cache lines.
constexpr int64_t delta_move_floats(int64_t kd) { return kd * kd + 32; }

struct DeltaArgs {
  DeltaOperand q, k, v, dy;
  const float* log_decay;  // [tokens, heads]
  const void* beta;        // [tokens, heads], I/O type
  float scale;
  const int32_t* cu;       // nullable: nseq sequences of seqlen tokens
  int64_t nseq, seqlen, tokens;
  int heads, kd, vd;
  int rep;                 // value heads per key head
  int64_t chunks;          // of all sequences; packed: at most so many
  int32_t per;             // chunks of a sequence (not packed)
  // packed: [nseq + 1] first chunk of each sequence, [nseq] their order and, with
  // spans, [nseq + 1] first span
  int32_t* table;
  uint8_t* record;         // [chunks, heads, delta_record]
  int back;                // with the backward's part of the records

  // span_chunks > 0: sequences in spans of so many chunks walked at the same time, not
  // packed `per_spans` to each, of all sequences at most `spans`; by span (all but each
  // sequence's last) and head the states that they end with, what they make of a state
  // (delta_move_floats, not the first) and for a backward the adjoints that enter them
  int span_chunks, per_spans, spans;
  float *span_ends, *span_moves, *span_backs;

  const float* s0;         // nullable; [nseq, heads, vd, kd]
  const float* ds_last;    // nullable
  void* o;                 // forward: [tokens, heads, vd]
  float* s_last;           // forward: nullable; [nseq, heads, vd, kd]

  // backward, all per chunk and head: state entering, adjoint leaving [vd, kd],
  // r and the adjoint of u [64, vd]
  float *states, *adjoints, *r, *y;
  void *dq, *dk, *dv;      // [tokens, key heads or heads, dim], I/O type
  float* dlog_decay;       // [tokens, heads]
  void* dbeta;             // [tokens, heads], I/O type
  float* ds0;              // nullable
};

hipError_t launch_delta_table(const DeltaArgs& a, hipStream_t stream);  // packed
hipError_t launch_delta_prep(const DeltaArgs& a, bool io_bf16, hipStream_t stream);
// The forward; with a.back the backward's two walks.
hipError_t launch_delta_walk_mm(const DeltaArgs& a, hipStream_t stream);   // bf16
hipError_t launch_delta_walk_f32(const DeltaArgs& a, hipStream_t stream);  // fp32
hipError_t launch_delta_span_states(const DeltaArgs& a, hipStream_t stream);
hipError_t launch_delta_grads(const DeltaArgs& a, bool io_bf16, hipStream_t stream);

struct DeltaStepArgs {
  float* h;             // [nslots, heads, vd, kd]
  const int32_t* slots; // nullable: row b uses slot b
  DeltaOperand q, k, v; // one token per row
  const float* log_decay;  // [batch, heads]
  const void* beta;        // [batch, heads], I/O type
  float scale;
  void* o;              // [batch, heads, vd]
  int64_t batch, nslots;
  int heads, kd, vd;
};
hipError_t launch_delta_step(const DeltaStepArgs& a, bool io_bf16, hipStream_t stream);

}  // namespace ssm
