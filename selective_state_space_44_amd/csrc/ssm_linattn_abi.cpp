// ssm_linattn_abi.cpp -- the extern "C" entry points of the linear attention
// with one decay per head and of the head norm with rotation (include/ssm.h):
// argument validation on the host before any HIP call, workspace carving and
// dispatch to the kernels.

#include "ssm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "ssm_launch.h"
#include "ssm_linattn.h"

namespace {

constexpr int64_t kMaxDim = 256;                  // channels of a head
constexpr int64_t kMaxHeads = 1 << 20;
// Elements between tokens: where a chunk of 64 tokens of one operand is addressed
// with 32-bit byte offsets, and where every token has a 64-bit address (no tensor
// on this card is larger).
constexpr int64_t kMaxStride = (int64_t)1 << 22;
constexpr int64_t kMaxFreeStride = (int64_t)1 << 38;
constexpr int64_t kMaxBlocks = INT32_MAX;

bool valid_dtype(int t) { return t == SSM_DTYPE_F32 || t == SSM_DTYPE_BF16; }
int64_t elem_bytes(int t) { return t == SSM_DTYPE_BF16 ? 2 : 4; }
int hip_status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }
bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename... P> bool all_aligned(P... p) { return (aligned(p) && ...); }

typedef std::initializer_list<const void*> Ptrs;

// No output (a non-null one) is an input or another output.
bool outputs_apart(Ptrs outs, Ptrs ins) {
  for (const void* const* o = outs.begin(); o != outs.end(); ++o) {
    if (!*o) continue;
    for (const void* i : ins)
      if (i == *o) return false;
    for (const void* const* p = outs.begin(); p != o; ++p)
      if (*p == *o) return false;
  }
  return true;
}

// Tokens `stride` elements apart, each holding heads * dim of them on a 16-byte
// boundary.
int check_stride(int64_t stride, int64_t heads, int64_t dim, int io_dtype,
                 int64_t most = kMaxStride) {
  if (stride < heads * dim || (stride * elem_bytes(io_dtype)) % 16 != 0) return SSM_ERR_INVALID_ARG;
  return stride > most ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

int check_free_stride(int64_t stride, int64_t heads, int64_t dim, int io_dtype) {
  return check_stride(stride, heads, dim, io_dtype, kMaxFreeStride);
}

bool valid_head_dim(int64_t d) { return d >= 8 && d <= kMaxDim && d % 8 == 0; }

struct LinSizes {
  int64_t batch, seqlen, nheads, nkvheads, kdim, vdim;
  bool packed;
  int64_t tokens() const { return packed ? seqlen : batch * seqlen; }
};

// Sizes shared by the whole-sequence entry points (SSM_OK: usable).
int check_sizes(const LinSizes& s, int io_dtype) {
  if (s.batch < 0 || s.seqlen < 0 || s.nheads < 0 || s.nkvheads < 0 || s.kdim <= 0 ||
      s.vdim <= 0 || !valid_dtype(io_dtype))
    return SSM_ERR_INVALID_ARG;
  if (s.nheads > 0 && (s.nkvheads == 0 || s.nheads % s.nkvheads != 0)) return SSM_ERR_INVALID_ARG;
  if (!valid_head_dim(s.kdim) || !valid_head_dim(s.vdim)) return SSM_ERR_UNSUPPORTED;
  // token numbers are 32-bit (cu_seqlens), and so are grid sizes
  if (s.nheads > kMaxHeads || s.batch > INT32_MAX || s.seqlen > INT32_MAX) return SSM_ERR_UNSUPPORTED;
  if (s.nheads * s.kdim > kMaxStride || s.nheads * s.vdim > kMaxStride) return SSM_ERR_UNSUPPORTED;
  // (the end of a chunk that the last token begins is a 32-bit number too)
  if (s.tokens() > INT32_MAX - (ssm::kLinChunk - 1)) return SSM_ERR_UNSUPPORTED;
  if (s.nheads > 0 && s.batch > kMaxBlocks / (s.nheads * 8)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

size_t align_up(size_t v) { return (v + 255) / 256 * 256; }

// How the sequences are cut.  A block walks a unit chunk by chunk, so a few
// long sequences are cut into segments.  A first launch gathers the state of
// each segment but the last, the states are joined along the sequence, and a
// second launch walks them; or (lead) the first launch walks the first segments
// beside the states of the others: 160 heads of 64 bf16 over 16384 tokens 418 us
// so, 501 without; 16 heads of 128 over 4096 63 so, 52 without.
struct LinPlan {
  bool lead;
  int64_t first_len;             // tokens of the first segment
  int64_t seg_len, segs, units;  // seg_len 0: a unit is a sequence
  int each;                      // packed: segments of every sequence; 0: of seg_len
  bool fold;                     // no join: every walk reads the states before its segment
};
// Packed, only the mean length is known here: one sequence much longer than the
// others is cut for the mean, or not at all (40 heads of 128, one of 16184 tokens
// among 200 of one: 1030 us, with 4 segments asked for 412).
constexpr int kBwdWalks = 3;  // dq, dk, dv
// whether the walk for the decay's gradient runs beside them
bool beside_of(const LinSizes& s, bool bf16, bool decay) {
  return decay && ssm::lin_decay_beside((int)s.kdim, (int)s.vdim, bf16);
}

// What a plan costs, in steps of one block alone on its CU over 64 tokens.  The
// constants are fits to timings of 4 to 400 heads of 64 and 128 over 256 to
// 16384 tokens, cut into 1 to 128 segments; they do not know the keys' size, and
// leave out how far the clock falls and what a launch's ends take (4 x 4096 x 40
// heads of 128: 171 us of steps, 241 in the launches).  A step takes 4.1 us at
// heads of 128 bf16, 2.6 at 64, 4.9 at 64 fp32; with the decay's gradient, where
// one walk is the long one, 12 and 4.2.  Both sides of it: 4 heads of 128 bf16
// over 16384 tokens 1035 us uncut, 69 in 64 segments; 256 heads over 4096 328
// uncut, 368 in two.
struct LinCost {
  double pair;   // a step where CUs have two blocks
  double round;  // a step of 512 blocks among more
  double pre;    // a state-only step
  double state;  // a block's state, written, joined and read
  double seg;    // a segment's part in the join, which is serial
};
constexpr LinCost kWideCost{1.65, 1.65, 0.4, 0.011, 0.08};   // 128 values to a block
constexpr LinCost kNarrowCost{1.4, 1.4, 0.4, 0.005, 0.08};  // 64
// with the decay's gradient
constexpr LinCost kWideDecayCost{1.33, 1.3, 0.25, 0.004, 0.03};
constexpr LinCost kNarrowDecayCost{1.3, 0.95, 0.15, 0.003, 0.03};
constexpr double kCutCost = 3.0;     // a launch or two more
constexpr double kLeadGain = 0.98;   // of the cost, for a lead to be taken
constexpr double kBesideCost = 1.2;  // a step of a walk beside states being gathered
// Bytes of states that a walk may read, one segment after the other, to join the
// segments before its own; above, a launch of its own joins them all.  160 heads
// of 128 in 3 segments 238 us folded, 257 not; in 4, 282 and 290; 16 heads in 6,
// 77 and 77; in 8, 70 and 64; 16 heads of 64 in 16, 32 and 35; in 32, 41 and 37.
constexpr int64_t kFoldBytes = 320 << 10;
constexpr int64_t kCus = 256;

// A step of n blocks.
double step_cost(const LinCost& c, bool decay, int64_t n) {
  const int64_t full = n / (2 * kCus), rest = n % (2 * kCus);
  if (decay && full > 0)  // blocks of uneven length fill each other's gaps
    return std::max(c.pair, c.round * n / (2 * kCus));
  return (rest == 0 ? 0.0 : rest <= kCus ? 1.0 : c.pair) + full * c.round;
}
// segs segments of `seg` chunks, states first.
double plain_cost(const LinCost& c, bool decay, int64_t blocks, int64_t seg, int64_t segs) {
  const double gather = c.pre * (double)((blocks * (segs - 1) + kCus - 1) / kCus);
  return seg * (gather + step_cost(c, decay, blocks * segs)) + kCutCost + c.state * blocks * segs +
         c.seg * segs;
}
// A first segment of `first` chunks in the lead of `rest` segments of `seg`.
double lead_cost(const LinCost& c, bool decay, int64_t blocks, int64_t first, int64_t seg,
                 int64_t rest) {
  const int64_t states = blocks * (rest - 1);
  // the first launch: as long as a first segment, or a state, or the work of both
  const double alone = first * (blocks + states <= kCus ? 1.0 : kBesideCost);
  const double gather = seg * c.pre * (double)((states + kCus - 1) / kCus);
  const double work = first * (double)blocks / (2 * kCus) * c.round +
                      seg * (double)states / kCus * c.pre;
  return std::max(alone, std::max(gather, work)) + seg * step_cost(c, decay, blocks * rest) +
         kCutCost + c.state * blocks * rest + c.seg * rest;
}

// For the forward, or the backward's walks (with the decay's gradient).
LinPlan lin_plan(const LinSizes& s, bool bf16, int nsplit, bool back, bool decay) {
  const int64_t T = s.tokens(), mean = s.batch > 0 ? (T + s.batch - 1) / s.batch : 0;
  const int64_t chunk = ssm::kLinChunk, chunks = (mean + chunk - 1) / chunk;
  int64_t segs = nsplit, first = 0, seg = 0;  // chunks
  bool lead = false;
  if (segs == 0) {
    const int64_t values = bf16 && s.vdim > 64 ? 128 : 64;
    // of one shape, in one launch; the decay's walk goes with the fuller plan
    const int64_t walks = !back ? 1 : beside_of(s, bf16, decay) ? kBwdWalks + 1
                          : s.kdim != s.vdim && !decay ? kBwdWalks - 1 : kBwdWalks;
    const int64_t blocks = s.batch * s.nheads * ((s.vdim + values - 1) / values) * walks;
    const LinCost& c = values == 128 ? (decay ? kWideDecayCost : kWideCost)
                                     : (decay ? kNarrowDecayCost : kNarrowCost);
    segs = 1;
    if (blocks < 2 * kCus) {
      double best = chunks * step_cost(c, decay, blocks), best_lead = best;
      int64_t lead_first = 0, lead_seg = 0, lead_rest = 0;
      for (int64_t n = 2; n <= chunks; n += 1 + n / 8) {
        if (c.state * blocks * n > best) break;
        const int64_t even = (chunks + n - 1) / n;
        const double plain = plain_cost(c, decay, blocks, even, (chunks + even - 1) / even);
        if (plain < best) best = plain, segs = n, first = seg = even;
        for (const double ratio : {0.7, 1.0, 1.4, 2.0}) {  // first to other segments
          const int64_t len = (int64_t)std::ceil(chunks / (n + ratio)), head = chunks - n * len;
          if (head < 1) continue;
          const double cost = lead_cost(c, decay, blocks, head, len, n);
          if (cost < best_lead) best_lead = cost, lead_first = head, lead_seg = len, lead_rest = n;
        }
      }
      // (the decay's walk alone is too long beside states being gathered)
      lead = best_lead < kLeadGain * best && (!decay || beside_of(s, bf16, decay));
      if (lead) segs = lead_rest + 1, first = lead_first, seg = lead_seg;
    }
  } else {
    seg = first = (chunks + segs - 1) / std::max<int64_t>(segs, 1);
  }
  const LinPlan uncut{false, 0, 0, 1, s.batch, 0, false};
  if (segs <= 1) return uncut;
  if (s.packed && nsplit) {  // as asked for, whatever the lengths are
    LinPlan p{false, chunk, chunk, 1, 0, 0, false};
    const int64_t most = T / chunk + 1;  // chunks of a sequence that holds all tokens
    p.each = (int)std::min(segs, most);
    p.units = std::min(s.batch * p.each, s.batch + T / chunk);
    p.fold = (p.each - 1) * s.kdim * s.vdim * 4 <= kFoldBytes;
    return p;
  }
  if (mean <= chunk) return uncut;
  LinPlan p{};
  p.lead = lead;
  p.first_len = first * chunk;
  p.seg_len = seg * chunk;
  p.segs = mean <= p.first_len ? 1 : 1 + (mean - p.first_len + p.seg_len - 1) / p.seg_len;
  // packed: at most one short segment and a first one to a sequence
  p.units = s.packed ? 2 * s.batch + T / p.seg_len : s.batch * p.segs;
  if (!s.packed && p.segs <= 1) return uncut;
  const int64_t before = s.packed ? T / p.seg_len + 1 : p.segs - 1;  // packed: all in one sequence
  p.fold = before * s.kdim * s.vdim * 4 <= kFoldBytes;
  return p;
}

// Workspace of a plan: the states between segments (of `states` walks) and,
// packed, the units.
struct PlanLayout {
  size_t state_off, state_bytes, table_off, total;
};
PlanLayout plan_layout(const LinSizes& s, const LinPlan& p, int states, size_t at) {
  PlanLayout l{at, 0, at, at};
  if (p.seg_len) l.state_bytes = align_up((size_t)p.units * s.nheads * s.kdim * s.vdim * 4);
  l.table_off = at + l.state_bytes * states;
  l.total = l.table_off +
            (s.packed ? align_up((size_t)ssm::lin_table_ints(p.units, s.batch) * 4) : 0);
  return l;
}

struct BwdLayout {
  size_t dk_off, dv_off, dg_off, total;
};
BwdLayout bwd_layout(const LinSizes& s, const LinPlan& p, bool bf16, bool dlog_decay) {
  BwdLayout l{};
  size_t at = 0;
  const bool shared = s.nheads != s.nkvheads;
  l.dk_off = at;
  if (shared) at += align_up((size_t)s.tokens() * s.nheads * s.kdim * 4);
  l.dv_off = at;
  if (shared) at += align_up((size_t)s.tokens() * s.nheads * s.vdim * 4);
  l.dg_off = at;
  if (dlog_decay)
    at += align_up((size_t)ssm::lin_dg_parts(p.units, (int)s.kdim, (int)s.vdim, bf16) * s.nheads * 4);
  l.total = at;
  return l;
}

// States between segments that are kept at once: one per walk, and two of the
// walk for the decay's gradient, which takes over the others' unless it runs
// beside them.
int bwd_states(const LinSizes& s, bool bf16, bool dlog_decay) {
  return beside_of(s, bf16, dlog_decay) ? kBwdWalks + 2 : kBwdWalks;
}

// n walks of one shape and plan.
hipError_t launch_walks(const ssm::LinArgs* walks, int n, bool bf16, hipStream_t stream) {
  return bf16 ? ssm::launch_linattn_mm(walks, n, stream) : ssm::launch_linattn_f32(walks, n, stream);
}

ssm::LinArgs base_args(const LinSizes& s, const int32_t* cu, const float* log_decay,
                       const LinPlan& p, const PlanLayout& l, char* ws) {
  ssm::LinArgs a{};
  a.log_decay = log_decay;
  a.cu = cu;
  a.nseq = s.batch;
  a.seqlen = s.seqlen;
  a.tokens = s.tokens();
  a.heads = (int)s.nheads;
  a.units = p.units;
  a.lead = p.lead;
  a.first_len = p.first_len;
  a.seg_len = p.seg_len;
  a.segs = p.segs;
  a.each = p.each;
  a.fold = p.fold;
  if (p.seg_len) a.ws_state = reinterpret_cast<float*>(ws + l.state_off);
  if (s.packed) a.unit_table = reinterpret_cast<int32_t*>(ws + l.table_off);
  return a;
}

}  // namespace

extern "C" {

int64_t ssm_linattn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int packed, int64_t nheads,
                                        int64_t nkvheads, int64_t kdim, int64_t vdim, int io_dtype,
                                        int nsplit) {
  const LinSizes s{batch, seqlen, nheads, nkvheads, kdim, vdim, packed != 0};
  if (check_sizes(s, io_dtype) != SSM_OK || nsplit < 0) return -1;
  if (batch == 0 || nheads == 0 || seqlen == 0) return 0;
  return (int64_t)plan_layout(s, lin_plan(s, io_dtype == SSM_DTYPE_BF16, nsplit, false, false), 1, 0)
      .total;
}

int ssm_linattn_fwd(int64_t batch, int64_t seqlen, const int32_t* cu_seqlens, int64_t nheads,
                    int64_t nkvheads, int64_t kdim, int64_t vdim, int io_dtype, const void* q,
                    int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, const float* log_decay, float scale, const float* h0,
                    void* o, float* h_last, int nsplit, void* workspace, size_t workspace_bytes,
                    void* stream) {
  const LinSizes s{batch, seqlen, nheads, nkvheads, kdim, vdim, cu_seqlens != nullptr};
  int st = check_sizes(s, io_dtype);
  if (st != SSM_OK) return st;
  if (nsplit < 0) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || nheads == 0) return SSM_OK;
  if (!log_decay) return SSM_ERR_INVALID_ARG;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (!all_aligned(h0, h_last) || (h_last && h_last == h0)) return SSM_ERR_INVALID_ARG;
  if (seqlen == 0) {
    if (!h_last) return SSM_OK;
    return hip_status(ssm::launch_copy_state(h0, h_last, batch * nheads * kdim * vdim, hs));
  }
  if (!q || !k || !v || !o) return SSM_ERR_INVALID_ARG;
  if (!all_aligned(q, k, v, o, workspace)) return SSM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(log_decay)) & 3u)
    return SSM_ERR_INVALID_ARG;
  if ((st = check_stride(q_stride, nheads, kdim, io_dtype)) != SSM_OK ||
      (st = check_stride(k_stride, nkvheads, kdim, io_dtype)) != SSM_OK ||
      (st = check_stride(v_stride, nkvheads, vdim, io_dtype)) != SSM_OK)
    return st;
  if (!outputs_apart({o, h_last, workspace}, {q, k, v, log_decay, h0, cu_seqlens}))
    return SSM_ERR_INVALID_ARG;
  const LinPlan plan = lin_plan(s, io_dtype == SSM_DTYPE_BF16, nsplit, false, false);
  const PlanLayout pl = plan_layout(s, plan, 1, 0);
  if (pl.total > 0 && (!workspace || workspace_bytes < pl.total)) return SSM_ERR_WORKSPACE;
  const int per = (int)(nheads / nkvheads);
  ssm::LinArgs a = base_args(s, cu_seqlens, log_decay, plan, pl, static_cast<char*>(workspace));
  if (ssm::launch_lin_units(a, hs) != hipSuccess) return SSM_ERR_HIP;
  a.q = {q, q_stride, 1};
  a.k = {k, k_stride, per};
  a.v = {v, v_stride, per};
  a.o = o;
  a.read_scale = a.pair_scale = scale;
  a.write_scale = 1.0f;
  a.s0 = h0;
  a.s_last = h_last;
  a.kd = (int)kdim;
  a.vd = (int)vdim;
  return hip_status(launch_walks(&a, 1, io_dtype == SSM_DTYPE_BF16, hs));
}

int64_t ssm_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int packed, int64_t nheads,
                                        int64_t nkvheads, int64_t kdim, int64_t vdim, int io_dtype,
                                        int need_dlog_decay, int nsplit) {
  const LinSizes s{batch, seqlen, nheads, nkvheads, kdim, vdim, packed != 0};
  if (check_sizes(s, io_dtype) != SSM_OK || nsplit < 0) return -1;
  if (batch == 0 || nheads == 0 || seqlen == 0) return 0;
  const LinPlan plan = lin_plan(s, io_dtype == SSM_DTYPE_BF16, nsplit, true,
                                need_dlog_decay != 0);
  const bool bf16 = io_dtype == SSM_DTYPE_BF16;
  const BwdLayout l = bwd_layout(s, plan, bf16, need_dlog_decay != 0);
  return (int64_t)plan_layout(s, plan, bwd_states(s, bf16, need_dlog_decay != 0), l.total).total;
}

int ssm_linattn_bwd(int64_t batch, int64_t seqlen, const int32_t* cu_seqlens, int64_t nheads,
                    int64_t nkvheads, int64_t kdim, int64_t vdim, int io_dtype, const void* q,
                    int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, const float* log_decay, float scale, const float* h0,
                    const void* dy, int64_t dy_stride, const float* dh_last, void* dq, void* dk,
                    void* dv, float* dlog_decay, float* dh0, int nsplit, void* workspace,
                    size_t workspace_bytes, void* stream) {
  const LinSizes s{batch, seqlen, nheads, nkvheads, kdim, vdim, cu_seqlens != nullptr};
  int st = check_sizes(s, io_dtype);
  if (st != SSM_OK) return st;
  if (nsplit < 0) return SSM_ERR_INVALID_ARG;
  if (nheads == 0) return SSM_OK;
  if (!log_decay) return SSM_ERR_INVALID_ARG;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (!all_aligned(h0, dh_last, dh0) || (reinterpret_cast<uintptr_t>(dlog_decay) & 3u) ||
      !outputs_apart({dh0, dlog_decay}, {h0, dh_last, log_decay}))
    return SSM_ERR_INVALID_ARG;
  if (batch == 0 || seqlen == 0) {  // no token: the final state is the given one
    if (dlog_decay) {
      const hipError_t e = ssm::launch_copy_state(nullptr, dlog_decay, nheads, hs);  // zeros
      if (e != hipSuccess) return SSM_ERR_HIP;
    }
    if (!dh0 || batch == 0) return SSM_OK;
    return hip_status(ssm::launch_copy_state(dh_last, dh0, batch * nheads * kdim * vdim, hs));
  }
  if (!q || !k || !v || !dy || !dq || !dk || !dv) return SSM_ERR_INVALID_ARG;
  if (!all_aligned(q, k, v, dy, dq, dk, dv, workspace)) return SSM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(log_decay)) & 3u)
    return SSM_ERR_INVALID_ARG;
  if ((st = check_stride(q_stride, nheads, kdim, io_dtype)) != SSM_OK ||
      (st = check_stride(k_stride, nkvheads, kdim, io_dtype)) != SSM_OK ||
      (st = check_stride(v_stride, nkvheads, vdim, io_dtype)) != SSM_OK ||
      (st = check_stride(dy_stride, nheads, vdim, io_dtype)) != SSM_OK)
    return st;
  if (!outputs_apart({dq, dk, dv, dlog_decay, dh0, workspace},
                     {q, k, v, log_decay, h0, dy, dh_last, cu_seqlens}))
    return SSM_ERR_INVALID_ARG;
  const LinPlan plan = lin_plan(s, io_dtype == SSM_DTYPE_BF16, nsplit, true,
                                dlog_decay != nullptr);
  const bool bf16 = io_dtype == SSM_DTYPE_BF16;
  const BwdLayout l = bwd_layout(s, plan, bf16, dlog_decay != nullptr);
  const PlanLayout pl =
      plan_layout(s, plan, bwd_states(s, bf16, dlog_decay != nullptr), l.total);
  if (pl.total > 0 && (!workspace || workspace_bytes < pl.total)) return SSM_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  const int per = (int)(nheads / nkvheads);
  const ssm::LinOperand Q{q, q_stride, 1}, K{k, k_stride, per}, V{v, v_stride, per},
      Y{dy, dy_stride, 1};
  const ssm::LinArgs base = base_args(s, cu_seqlens, log_decay, plan, pl, ws);
  if (ssm::launch_lin_units(base, hs) != hipSuccess) return SSM_ERR_HIP;

  auto state_of = [&](ssm::LinArgs& a, int walk) {
    if (plan.seg_len) a.ws_state = reinterpret_cast<float*>(ws + pl.state_off + walk * pl.state_bytes);
  };
  ssm::LinArgs walks[kBwdWalks + 1] = {base, base, base, base};
  {
    ssm::LinArgs& a = walks[0];  // dq_t = scale sum_{s<=t} a^(t-s) (dy_t . v_s) k_s + ...
    a.q = Y, a.k = V, a.v = K;
    a.kd = (int)vdim, a.vd = (int)kdim;
    a.read_scale = a.pair_scale = scale, a.write_scale = 1.0f;
    a.s0 = h0, a.s0_swap = 1;
    a.o = dq;
  }
  {
    ssm::LinArgs& a = walks[1];  // dk_s = scale sum_{t>=s} a^(t-s) (v_s . dy_t) q_t + ...
    a.rev = 1;
    a.q = V, a.k = Y, a.v = Q;
    a.kd = (int)vdim, a.vd = (int)kdim;
    a.read_scale = 1.0f, a.pair_scale = a.write_scale = scale;
    a.s0 = dh_last, a.s0_swap = 1;
    a.o = per > 1 ? static_cast<void*>(ws + l.dk_off) : dk;
    a.o_f32 = per > 1;
    state_of(a, 1);
  }
  {
    ssm::LinArgs& a = walks[2];  // dv_s = scale sum_{t>=s} a^(t-s) (k_s . q_t) dy_t
    a.rev = 1;                   //        + a^(L-1-s) dh_last k_s
    a.q = K, a.k = Q, a.v = Y;
    a.kd = (int)kdim, a.vd = (int)vdim;
    a.read_scale = 1.0f, a.pair_scale = a.write_scale = scale;
    a.s0 = dh_last;
    a.s_last = dh0;
    a.o = per > 1 ? static_cast<void*>(ws + l.dv_off) : dv;
    a.o_f32 = per > 1;
    state_of(a, 2);
  }
  const bool beside = beside_of(s, bf16, dlog_decay != nullptr);
  if (dlog_decay) {
    ssm::LinArgs& a = walks[3];  // sum over t of dy_t . do_t / dg
    a.q = Q, a.k = K, a.v = V;
    a.kd = (int)kdim, a.vd = (int)vdim;
    a.read_scale = a.pair_scale = scale, a.write_scale = 1.0f;
    a.s0 = h0;
    a.dy = Y;
    a.ds_last = dh_last;
    a.dg_part = reinterpret_cast<float*>(ws + l.dg_off);
    const int first = beside ? kBwdWalks : 0;
    state_of(a, first);
    if (plan.seg_len) a.ws_tangent = a.ws_state + pl.state_bytes / sizeof(float);
  }
  // one launch for the walks of one shape
  const int together = kdim != vdim ? 2 : beside ? 4 : 3;
  if (launch_walks(walks, together, bf16, hs) != hipSuccess) return SSM_ERR_HIP;
  if (together == 2 && launch_walks(walks + 2, beside ? 2 : 1, bf16, hs) != hipSuccess)
    return SSM_ERR_HIP;
  if (dlog_decay && !beside && launch_walks(walks + 3, 1, bf16, hs) != hipSuccess)
    return SSM_ERR_HIP;
  if (per == 1 && !dlog_decay) return SSM_OK;
  ssm::LinSums sums{};
  if (per > 1) {
    const int64_t rows = s.tokens() * nkvheads;
    sums.k = {reinterpret_cast<float*>(ws + l.dk_off), dk, rows * kdim, (int)kdim};
    sums.v = {reinterpret_cast<float*>(ws + l.dv_off), dv, rows * vdim, (int)vdim};
    sums.per = per;
    sums.kvheads = (int)nkvheads;
    if (s.packed)
      sums.held = base.unit_table + ssm::lin_table_ints(plan.units, batch) - 2;
  }
  if (dlog_decay) {
    sums.dg_part = walks[3].dg_part;
    sums.dg = dlog_decay;
    sums.parts = ssm::lin_dg_parts(plan.units, (int)kdim, (int)vdim, bf16);
    sums.heads = (int)nheads;
  }
  return hip_status(ssm::launch_closing_sums(sums, bf16, hs));
}

int ssm_linattn_step(int64_t batch, int64_t nslots, const int32_t* slots, int64_t nheads,
                     int64_t nkvheads, int64_t kdim, int64_t vdim, int io_dtype, float* h,
                     const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                     const void* v, int64_t v_stride, const float* log_decay, float scale, void* o,
                     void* stream) {
  const LinSizes s{batch, 1, nheads, nkvheads, kdim, vdim, false};
  int st = check_sizes(s, io_dtype);
  if (st != SSM_OK) return st;
  if (nslots < 0 || (!slots && nslots < batch)) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || nheads == 0) return SSM_OK;
  if (!h || !q || !k || !v || !log_decay || !o) return SSM_ERR_INVALID_ARG;
  if (!all_aligned(h, q, k, v, o)) return SSM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(slots) | reinterpret_cast<uintptr_t>(log_decay)) & 3u)
    return SSM_ERR_INVALID_ARG;
  if ((st = check_free_stride(q_stride, nheads, kdim, io_dtype)) != SSM_OK ||
      (st = check_free_stride(k_stride, nkvheads, kdim, io_dtype)) != SSM_OK ||
      (st = check_free_stride(v_stride, nkvheads, vdim, io_dtype)) != SSM_OK)
    return st;
  if (!outputs_apart({h, o}, {q, k, v, log_decay, slots})) return SSM_ERR_INVALID_ARG;
  ssm::LinStepArgs a{};
  const int per = (int)(nheads / nkvheads);
  a.h = h;
  a.slots = slots;
  a.q = {q, q_stride, 1};
  a.k = {k, k_stride, per};
  a.v = {v, v_stride, per};
  a.log_decay = log_decay;
  a.scale = scale;
  a.o = o;
  a.batch = batch;
  a.nslots = nslots;
  a.heads = (int)nheads;
  a.kd = (int)kdim;
  a.vd = (int)vdim;
  return hip_status(
      ssm::launch_linattn_step(a, io_dtype == SSM_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Sizes and inputs shared by the norm-and-rotation's two directions.
int check_rotate(int64_t tokens, int64_t seqlen, int64_t nq, int64_t nk, int64_t dim, int64_t rot,
                 int interleaved, int io_dtype, float eps, int64_t npos) {
  if (tokens < 0 || seqlen < 0 || nq < 0 || nk < 0 || dim <= 0 || rot < 0 || rot > dim ||
      npos < 0 || !valid_dtype(io_dtype) || (interleaved != 0 && interleaved != 1) || !(eps >= 0.0f))
    return SSM_ERR_INVALID_ARG;
  if (!valid_head_dim(dim) || rot % 4 != 0) return SSM_ERR_UNSUPPORTED;
  if (nq > kMaxStride / dim || nk > kMaxStride / dim) return SSM_ERR_UNSUPPORTED;
  // the grid holds a block for every 256 / 64 pairs of rows
  if (tokens > 0 && tokens > INT32_MAX / (nq + nk + 2)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

int rotate_inputs(ssm::RotateArgs& a, int64_t tokens, int64_t seqlen, int64_t nq, int64_t nk,
                  int64_t dim, int64_t rot, int interleaved, int io_dtype, const void* q,
                  int64_t q_stride, const void* k, int64_t k_stride, const float* cos,
                  const float* sin, int64_t npos, const int64_t* positions, const float* qw,
                  const float* kw, float eps) {
  if ((nq > 0 && !q) || (nk > 0 && !k)) return SSM_ERR_INVALID_ARG;
  if (rot > 0) {
    if (!cos || !sin) return SSM_ERR_INVALID_ARG;
    // without positions token t stands at t % seqlen, which has to be in the table
    if (!positions && (seqlen == 0 || seqlen > npos)) return SSM_ERR_INVALID_ARG;
  }
  if (!all_aligned(q, k, cos, sin, qw, kw) || (reinterpret_cast<uintptr_t>(positions) & 7u))
    return SSM_ERR_INVALID_ARG;
  int st;
  if (nq > 0 && (st = check_free_stride(q_stride, nq, dim, io_dtype)) != SSM_OK) return st;
  if (nk > 0 && (st = check_free_stride(k_stride, nk, dim, io_dtype)) != SSM_OK) return st;
  a.x[0] = q, a.x[1] = k;
  a.stride[0] = q_stride, a.stride[1] = k_stride;
  a.w[0] = qw, a.w[1] = kw;
  a.cos = cos, a.sin = sin;
  a.positions = positions;
  a.tokens = tokens, a.npos = npos;
  a.seqlen = (uint32_t)std::min(seqlen > 0 ? seqlen : 1, tokens);
  a.heads[0] = (int)nq, a.heads[1] = (int)nk;
  a.dim = (int)dim, a.rot = (int)rot;
  a.interleaved = interleaved;
  a.eps = eps;
  return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_qk_norm_rotate_fwd(int64_t tokens, int64_t seqlen, int64_t nqheads, int64_t nkheads,
                           int64_t headdim, int64_t rotdim, int interleaved, int io_dtype,
                           const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const float* cos, const float* sin, int64_t npos,
                           const int64_t* positions, const float* q_weight, const float* k_weight,
                           float eps, void* q_out, void* k_out, void* stream) {
  int st = check_rotate(tokens, seqlen, nqheads, nkheads, headdim, rotdim, interleaved, io_dtype,
                        eps, npos);
  if (st != SSM_OK) return st;
  if (tokens == 0 || nqheads + nkheads == 0) return SSM_OK;
  ssm::RotateArgs a{};
  st = rotate_inputs(a, tokens, seqlen, nqheads, nkheads, headdim, rotdim, interleaved, io_dtype, q,
                     q_stride, k, k_stride, cos, sin, npos, positions, q_weight, k_weight, eps);
  if (st != SSM_OK) return st;
  if ((nqheads > 0 && !q_out) || (nkheads > 0 && !k_out)) return SSM_ERR_INVALID_ARG;
  if (!all_aligned(q_out, k_out) ||
      !outputs_apart({q_out, k_out}, {q, k, cos, sin, positions, q_weight, k_weight}))
    return SSM_ERR_INVALID_ARG;
  a.out[0] = q_out, a.out[1] = k_out;
  return hip_status(
      ssm::launch_rotate_fwd(a, io_dtype == SSM_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

int64_t ssm_qk_norm_rotate_bwd_workspace_bytes(int64_t tokens, int64_t nqheads, int64_t nkheads,
                                               int64_t headdim) {
  if (check_rotate(tokens, 0, nqheads, nkheads, headdim, 0, 0, SSM_DTYPE_F32, 0.0f, 0) != SSM_OK)
    return -1;
  return (int64_t)ssm::rotate_bwd_blocks(tokens, (int)(nqheads + nkheads), (int)headdim) *
         headdim * 4;
}

int ssm_qk_norm_rotate_bwd(int64_t tokens, int64_t seqlen, int64_t nqheads, int64_t nkheads,
                           int64_t headdim, int64_t rotdim, int interleaved, int io_dtype,
                           const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const float* cos, const float* sin, int64_t npos,
                           const int64_t* positions, const float* q_weight, const float* k_weight,
                           float eps, const void* dq_out, int64_t dq_out_stride,
                           const void* dk_out, int64_t dk_out_stride, void* dq, void* dk,
                           float* dq_weight, float* dk_weight, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int st = check_rotate(tokens, seqlen, nqheads, nkheads, headdim, rotdim, interleaved, io_dtype,
                        eps, npos);
  if (st != SSM_OK) return st;
  const bool weights = dq_weight || dk_weight;
  const bool none = tokens == 0 || nqheads + nkheads == 0;
  if (none && !weights) return SSM_OK;
  ssm::RotateArgs a{};
  if (!none) {
    st = rotate_inputs(a, tokens, seqlen, nqheads, nkheads, headdim, rotdim, interleaved, io_dtype,
                       q, q_stride, k, k_stride, cos, sin, npos, positions, q_weight, k_weight,
                       eps);
    if (st != SSM_OK) return st;
    if ((nqheads > 0 && (!dq_out || !dq)) || (nkheads > 0 && (!dk_out || !dk)))
      return SSM_ERR_INVALID_ARG;
    if (nqheads > 0 && (st = check_free_stride(dq_out_stride, nqheads, headdim, io_dtype)) != SSM_OK)
      return st;
    if (nkheads > 0 && (st = check_free_stride(dk_out_stride, nkheads, headdim, io_dtype)) != SSM_OK)
      return st;
  }
  if (!all_aligned(dq_out, dk_out, dq, dk, workspace) || ((reinterpret_cast<uintptr_t>(dq_weight) |
      reinterpret_cast<uintptr_t>(dk_weight)) & 3u) ||
      !outputs_apart({dq, dk, dq_weight, dk_weight, workspace},
                     {q, k, cos, sin, positions, q_weight, k_weight, dq_out, dk_out}))
    return SSM_ERR_INVALID_ARG;
  if (weights) {
    const size_t need =
        (size_t)ssm_qk_norm_rotate_bwd_workspace_bytes(tokens, nqheads, nkheads, headdim);
    if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
    a.dw_part = static_cast<float*>(workspace);
    a.dw[0] = dq_weight, a.dw[1] = dk_weight;
  }
  a.dim = (int)headdim;
  a.rot = (int)rotdim;
  a.dy[0] = dq_out, a.dy[1] = dk_out;
  a.dstride[0] = dq_out_stride, a.dstride[1] = dk_out_stride;
  a.out[0] = dq, a.out[1] = dk;
  return hip_status(
      ssm::launch_rotate_bwd(a, io_dtype == SSM_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
