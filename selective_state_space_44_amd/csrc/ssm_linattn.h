// ssm_linattn.h -- internal interface between the C ABI (ssm_linattn_abi.cpp)
// and the kernels of the linear attention with one decay per head
// (ssm_linattn*.hip) and of the head norm with rotation (ssm_rotate.hip).
// Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

// Blocks of so many threads that a launch may have: a grid's threads are counted
// in 32 bits.  Larger ones go in slices.
constexpr uint32_t max_blocks(uint32_t threads) { return UINT32_MAX / threads; }

// One token-major operand [tokens, heads / hdiv, dim]: element (t, h, d) is at
// t * stride + (h / hdiv) * dim + d.
struct LinOperand {
  const void* p;
  int64_t stride;  // elements between tokens
  int hdiv;        // query heads per head of this operand
};

// One walk over every sequence.  The forward computes, per head,
//   o_t = sum over s <= t of a^(t-s) (q_t . k_s) v_s  +  a^(t+1) S0 q_t.
// The backward is the same sum with the operands' roles exchanged:
//   dq: (q, k, v) := (dy, v, k), state S0^T;
//   dv: (k, q, dy), dk: (v, dy, q), both from the last token back (rev).
// Backwards in time the given state is dh_last, which the last token reads
// undecayed: reads decay by one step less and writes by one step more.
struct LinArgs {
  LinOperand q, k, v;
  void* o;              // [tokens, heads, vd]
  const float* log_decay;  // [heads]
  float read_scale;     // of S q
  float pair_scale;     // of (q . k)
  float write_scale;    // of v k^T on its way into the state
  const float* s0;      // nullable; [nseq, heads, vd, kd], or [nseq, heads, kd, vd] when s0_swap
  int s0_swap;
  float* s_last;        // nullable; [nseq, heads, vd, kd]
  const int32_t* cu;    // nullable: nseq sequences of seqlen tokens
  int64_t nseq, seqlen, tokens;
  int heads, kd, vd;
  int rev;
  int o_f32;            // o in fp32 whatever the operands' type
  // Derivative by the log decay: with dg_part given the walk carries dS/dg as
  // well and writes, instead of o and s_last, its part of
  //   sum over t of dy_t . do_t/dg  +  <ds_last, dS_last/dg>
  // per block, [lin_dg_parts(..), heads].
  float* dg_part;
  LinOperand dy;        // [tokens, heads, vd]
  const float* ds_last; // nullable; [nseq, heads, vd, kd]
  int64_t units;        // launched per head; packed: at most so many
  int64_t first_len;    // of a sequence's first segment, seg_len of the others
  int lead;             // first segments are walked in the first launch
  int64_t seg_len, segs;
  int each;             // packed: 0, or a sequence's segments, of its own length (seg_len unused)
  int fold;             // the walks join the states of the segments before them themselves
  int32_t* unit_table;  // packed
  float* ws_state;      // [units, heads, vd, kd] when cut into segments
  float* ws_tangent;    // likewise, with dg_part
};

// Work of the chunked walks: unit u of a head is a sequence (seg_len 0) or a
// segment of one (whole chunks: first_len tokens, then seg_len each, the last
// one what is left; with `each`, all of one length), run by a block of its own.  Sequences of one length have
// `segs` segments each; the units of packed ones stand in unit_table, written by
// launch_lin_units:
//   [0] their number, [1 + 2u] sequence and segment of unit u,
//   [1 + 2 units + n] first unit of sequence n,
//   [1 + 2 units + nseq] first token of any sequence and the end of the last.
// ws_state holds each unit's end state (that of a segment past the first without
// what came before it); without fold, after the join, the state entering it.
constexpr int kLinChunk = 64;
constexpr int64_t lin_table_ints(int64_t units, int64_t nseq) { return 3 + 2 * units + nseq; }

int64_t lin_dg_parts(int64_t units, int kd, int vd, bool io_bf16);
hipError_t launch_lin_units(const LinArgs& a, hipStream_t stream);
// n <= 3 walks of one head's sizes (kd, vd) and plan.  One with dg_part goes
// alone, but as a last one beside the others where lin_decay_beside says so.
bool lin_decay_beside(int kd, int vd, bool io_bf16);
hipError_t launch_linattn_mm(const LinArgs* walks, int n, hipStream_t stream);   // bf16
hipError_t launch_linattn_f32(const LinArgs* walks, int n, hipStream_t stream);  // fp32

// The backward's closing sums, each in a fixed order:
//   out[t, g, d] = sum over the `per` query heads h of key head g of in[t, h, d]
// (fp32 in; out in the I/O type; count elements of out, none to leave out), and
//   dg[h] = sum over parts of dg_part[i, h]  (dg null to leave out).
struct LinGroupSum {
  const float* in;
  void* out;
  int64_t count;
  int dim;
};
struct LinSums {
  LinGroupSum k, v;
  int per;
  const int32_t* held;  // nullable: the tokens held[0] .. held[1] - 1 have a sum, the others none
  int kvheads;
  const float* dg_part;
  float* dg;
  int64_t parts;
  int heads;
};
hipError_t launch_closing_sums(const LinSums& a, bool io_bf16, hipStream_t stream);

struct LinStepArgs {
  float* h;             // [nslots, heads, vd, kd]
  const int32_t* slots; // nullable: row b uses slot b
  LinOperand q, k, v;   // one token per row
  const float* log_decay;
  float scale;
  void* o;              // [batch, heads, vd]
  int64_t batch, nslots;
  int heads, kd, vd;
};
hipError_t launch_linattn_step(const LinStepArgs& a, bool io_bf16, hipStream_t stream);

struct RotateArgs {
  const void* x[2];     // q, k: [tokens, heads[i], dim], tokens stride[i] apart
  int64_t stride[2];
  const void* dy[2];    // backward only: gradients of the outputs
  int64_t dstride[2];
  void* out[2];         // forward: outputs; backward: dq, dk (contiguous)
  const float* w[2];    // nullable
  const float* cos;     // [npos, rot / 2]
  const float* sin;
  const int64_t* positions;  // nullable: t % seqlen
  float* dw_part;       // backward: [blocks, dim] partial weight gradients, nullable
  float* dw[2];         // nullable
  int64_t tokens, npos;
  uint32_t seqlen;      // of every sequence; `tokens` where that is less
  int heads[2];
  int dim, rot;
  int interleaved;
  float eps;
};
hipError_t launch_rotate_fwd(const RotateArgs& a, bool io_bf16, hipStream_t stream);
hipError_t launch_rotate_bwd(const RotateArgs& a, bool io_bf16, hipStream_t stream);
int rotate_bwd_blocks(int64_t tokens, int heads, int dim);

}  // namespace ssm
