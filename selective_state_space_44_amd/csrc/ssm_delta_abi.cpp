// ssm_delta_abi.cpp -- the extern "C" entry points of the gated delta rule and of
// the layer norm (include/ssm.h): argument validation on the host before any HIP
// call, workspace carving and dispatch to the kernels.

#include "ssm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "ssm_checks.h"
#include "ssm_delta.h"
#include "ssm_launch.h"
#include "ssm_norm.h"

namespace {

using namespace ssm;

// Channels of a head: a chunk's keys and queries, all their channels, and its
// triangles stand in LDS at once (fp32: 128 KB of 160 with 128 channels); values go
// by blocks.
constexpr int64_t kMaxKeys = 128, kMaxValues = 256;

struct DeltaSizes {
  int64_t batch, seqlen, heads, kheads, kdim, vdim;
  bool packed;
  int64_t tokens() const { return packed ? seqlen : batch * seqlen; }
  int64_t per() const { return (seqlen + kDeltaChunk - 1) / kDeltaChunk; }
  // packed: a short chunk to every sequence at most
  int64_t chunks() const { return packed ? seqlen / kDeltaChunk + batch : batch * per(); }
  int64_t state() const { return kdim * vdim; }
};

int check_sizes(const DeltaSizes& s, int io_dtype) {
  if (s.batch < 0 || s.seqlen < 0 || s.heads < 0 || s.kheads < 0 || s.kdim <= 0 || s.vdim <= 0 ||
      !valid_dtype(io_dtype))
    return SSM_ERR_INVALID_ARG;
  if (s.heads > 0 && (s.kheads == 0 || s.heads % s.kheads != 0)) return SSM_ERR_INVALID_ARG;
  if (s.kdim % 8 || s.vdim % 8 || s.kdim > kMaxKeys || s.vdim > kMaxValues)
    return SSM_ERR_UNSUPPORTED;
  // token numbers are 32-bit (cu_seqlens), and so is the end of a chunk that the
  // last token begins
  if (s.heads > kMaxHeads || s.batch > INT32_MAX || s.seqlen > INT32_MAX ||
      s.tokens() > INT32_MAX - (kDeltaChunk - 1))
    return SSM_ERR_UNSUPPORTED;
  if (s.heads * s.kdim > kMaxStride || s.heads * s.vdim > kMaxStride) return SSM_ERR_UNSUPPORTED;
  if (s.heads > 0 && s.batch > kMaxBlocks / (s.heads * 8)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Spans that the sequences' walks are cut in (ssm_delta_walk.h), of how many chunks: as
// many as give every CU its blocks in the first launch.  With spans and without, one
// sequence of bf16 heads of 128 x 128: 32 heads over 65536 tokens 2.38 and 4.63 ms, 8 over
// 32768 0.39 and 2.19, 16 over 2048 79 and 152 us; in three 64 heads over 16384 1020 and
// 1253.  A backward's blocks are twice as many from the start: 8 heads over 32768 tokens
// 1.11 and 3.24 ms, 32 over 16384 1.82 and 2.31; in three 48 over 4096 732 and 721 us, so
// it takes four or none.  Spans of two chunks at least: 8 heads over 1024 tokens take 83 us
// in one, 63 in spans of four chunks, 56 of two; 72 fp32 heads of 64 over 517 tokens 78 in
// one and 77.  Of three in a backward, where those of two pay for few heads only: 8 over
// 1024 128 in one, 102 of three and 91 of two, but 24 over 512 87 in one and 99 of two.  Of
// packed sequences the host knows the mean length only.  The longer ones are cut into
// more, so two spans on average pay, of a backward three: 3 of 16384 tokens in all and 8
// heads 219 and 956 us, 32 heads 681 and 1020, 24 of 8 heads of 128 x 64 152 and 186;
// backward 624 and 1449 us of the first.
//
// The states are taken from span to span one after the other, so of one or two heads
// more spans than walks would use cost more there: n spans take J n + 2 K m / n for m
// chunks of K, least at n^2 = (2 K / J) m.  One sequence of 32768 tokens and one head,
// bf16, 128 x 128, of 128, 48 and 24 spans 321, 210 and 255 us, its backward (of 86, 48
// and 24) 376, 306 and 350; 64 x 64 of 256, 64 and 24 179, 110 and 179, fp32 of 256, 96
// and 48 196, 148 and 187; two heads of 128 over 16384 of 64, 32 and 16 192, 155 and 189.
struct Spans {
  int chunks = 0, per = 0;  // of a span; not packed: spans of a sequence
  int64_t count = 0;        // at most so many
};
Spans spans_of(const DeltaSizes& s, bool back, int io_dtype) {
  // (of fp32 keys of 128 a CU holds one)
  const int64_t most = io_dtype == SSM_DTYPE_F32 && s.kdim > 64 ? 256 : 512;
  const int64_t wide = s.vdim <= 32 ? 32 : 64, units = s.batch * s.heads;
  const int64_t v = units * ((s.vdim + wide - 1) / wide) * (back ? 2 : 1),
                k = units * ((s.kdim + wide - 1) / wide);
  const int64_t least = back ? 3 : 2, few = (back ? 4 : 3) - (s.packed ? 1 : 0);
  // v (n - 1) + k (n - 2) blocks for n spans a sequence, of packed ones on average
  const int64_t chunks = s.chunks(), mean = chunks / s.batch;
  const int64_t join = (s.kdim > 64 ? 4 : 12) * (io_dtype == SSM_DTYPE_F32 ? 2 : 1);
  const int64_t n = std::min({(most + v + 2 * k) / (v + k), mean / least,
                              (int64_t)std::sqrt((double)(join * mean))});
  Spans r;
  if (n < few) return r;
  r.chunks = (int)((mean + n - 1) / n);
  r.per = (int)((s.per() + r.chunks - 1) / r.chunks);
  r.count = s.packed ? chunks / r.chunks + s.batch : s.batch * r.per;
  return r;
}

struct DeltaLayout {
  size_t span_ends, span_moves, span_backs, record, states, adjoints, r, y, total;
};
DeltaLayout layout_of(const DeltaSizes& s, bool back, int io_dtype) {
  DeltaLayout l{};
  const size_t units = (size_t)s.chunks() * s.heads;
  size_t at = s.packed ? align_up((size_t)(3 * s.batch + 2) * 4) : 0;
  auto take = [&](size_t floats) {
    const size_t here = at;
    at += align_up(floats * 4);
    return here;
  };
  l.record = take(units * (size_t)delta_record(back).size / 4);
  const Spans cut = spans_of(s, back, io_dtype);
  if (cut.chunks > 0) {
    const size_t spans = (size_t)((cut.count - s.batch) * s.heads);
    l.span_ends = take(spans * s.state());
    l.span_moves = take(spans * (size_t)delta_move_floats(s.kdim));
    if (back) l.span_backs = take(spans * s.state());
  }
  if (back) {
    l.states = take(units * s.state());
    l.adjoints = take(units * s.state());
    l.r = take(units * kDeltaChunk * s.vdim);
    l.y = take(units * kDeltaChunk * s.vdim);
  }
  l.total = at;
  return l;
}

DeltaArgs delta_args(const DeltaSizes& s, const int32_t* cu, const void* q, int64_t q_stride,
                     const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                     const float* log_decay, const void* beta, float scale, const float* h0,
                     const DeltaLayout& l, void* workspace, bool back, int io_dtype) {
  DeltaArgs a{};
  const int rep = (int)(s.heads / s.kheads);
  char* ws = static_cast<char*>(workspace);
  a.q = {q, q_stride, rep};
  a.k = {k, k_stride, rep};
  a.v = {v, v_stride, 1};
  a.log_decay = log_decay;
  a.beta = beta;
  a.scale = scale;
  a.cu = cu;
  a.nseq = s.batch;
  a.seqlen = s.seqlen;
  a.tokens = s.tokens();
  a.heads = (int)s.heads;
  a.kd = (int)s.kdim;
  a.vd = (int)s.vdim;
  a.rep = rep;
  a.chunks = s.chunks();
  a.per = (int32_t)s.per();
  a.back = back;
  a.s0 = h0;
  if (s.packed) a.table = reinterpret_cast<int32_t*>(ws);
  auto floats = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  a.record = reinterpret_cast<uint8_t*>(ws + l.record);
  const Spans spans = spans_of(s, back, io_dtype);
  a.span_chunks = spans.chunks;
  a.per_spans = spans.per;
  a.spans = (int)spans.count;
  if (spans.chunks > 0) {
    a.span_ends = floats(l.span_ends);
    a.span_moves = floats(l.span_moves);
    if (back) a.span_backs = floats(l.span_backs);
  }
  if (back) {
    a.states = floats(l.states);
    a.adjoints = floats(l.adjoints);
    a.r = floats(l.r);
    a.y = floats(l.y);
  }
  return a;
}

// What the whole-sequence calls check of their inputs (there are tokens).
int check_inputs(const DeltaSizes& s, int io_dtype, const int32_t* cu, const void* q,
                 int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 const float* log_decay, const void* beta) {
  if (!q || !k || !v || !log_decay || !beta) return SSM_ERR_INVALID_ARG;
  if (!all_aligned(q, k, v) || !aligned(cu, 4) || !aligned(log_decay, 4) ||
      !aligned(beta, (unsigned)elem_bytes(io_dtype)))
    return SSM_ERR_INVALID_ARG;
  int st;
  if ((st = check_stride(q_stride, s.kheads, s.kdim, io_dtype)) != SSM_OK ||
      (st = check_stride(k_stride, s.kheads, s.kdim, io_dtype)) != SSM_OK ||
      (st = check_stride(v_stride, s.heads, s.vdim, io_dtype)) != SSM_OK)
    return st;
  return SSM_OK;
}

hipError_t launch_walk(const DeltaArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_delta_walk_mm(a, stream) : launch_delta_walk_f32(a, stream);
}

}  // namespace

extern "C" {

int64_t ssm_delta_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int packed, int64_t nheads,
                                      int64_t nkheads, int64_t kdim, int64_t vdim, int io_dtype) {
  const DeltaSizes s{batch, seqlen, nheads, nkheads, kdim, vdim, packed != 0};
  if (check_sizes(s, io_dtype) != SSM_OK) return -1;
  if (batch == 0 || nheads == 0 || seqlen == 0) return 0;
  return (int64_t)layout_of(s, false, io_dtype).total;
}

int ssm_delta_fwd(int64_t batch, int64_t seqlen, const int32_t* cu_seqlens, int64_t nheads,
                  int64_t nkheads, int64_t kdim, int64_t vdim, int io_dtype, const void* q,
                  int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  const float* log_decay, const void* beta, float scale, const float* h0, void* o,
                  float* h_last, void* workspace, size_t workspace_bytes, void* stream) {
  const DeltaSizes s{batch, seqlen, nheads, nkheads, kdim, vdim, cu_seqlens != nullptr};
  int st = check_sizes(s, io_dtype);
  if (st != SSM_OK) return st;
  if (batch == 0 || nheads == 0) return SSM_OK;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (!all_aligned(h0, h_last) || (h_last && h_last == h0)) return SSM_ERR_INVALID_ARG;
  if (seqlen == 0) {
    if (!h_last) return SSM_OK;
    return hip_status(launch_copy_state(h0, h_last, batch * nheads * s.state(), hs));
  }
  st = check_inputs(s, io_dtype, cu_seqlens, q, q_stride, k, k_stride, v, v_stride, log_decay, beta);
  if (st != SSM_OK) return st;
  if (!o || !all_aligned(o, workspace) ||
      !outputs_apart({o, h_last, workspace}, {q, k, v, log_decay, beta, h0, cu_seqlens}))
    return SSM_ERR_INVALID_ARG;
  const DeltaLayout l = layout_of(s, false, io_dtype);
  if (!workspace || workspace_bytes < l.total) return SSM_ERR_WORKSPACE;
  const bool bf16 = io_dtype == SSM_DTYPE_BF16;
  DeltaArgs a = delta_args(s, cu_seqlens, q, q_stride, k, k_stride, v, v_stride, log_decay, beta,
                           scale, h0, l, workspace, false, io_dtype);
  a.o = o;
  a.s_last = h_last;
  hipError_t e = launch_delta_table(a, hs);
  if (e == hipSuccess) e = launch_delta_prep(a, bf16, hs);
  if (e == hipSuccess) e = launch_walk(a, bf16, hs);
  return hip_status(e);
}

int64_t ssm_delta_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int packed, int64_t nheads,
                                      int64_t nkheads, int64_t kdim, int64_t vdim, int io_dtype) {
  const DeltaSizes s{batch, seqlen, nheads, nkheads, kdim, vdim, packed != 0};
  if (check_sizes(s, io_dtype) != SSM_OK) return -1;
  if (batch == 0 || nheads == 0 || seqlen == 0) return 0;
  return (int64_t)layout_of(s, true, io_dtype).total;
}

int ssm_delta_bwd(int64_t batch, int64_t seqlen, const int32_t* cu_seqlens, int64_t nheads,
                  int64_t nkheads, int64_t kdim, int64_t vdim, int io_dtype, const void* q,
                  int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  const float* log_decay, const void* beta, float scale, const float* h0,
                  const void* dy, int64_t dy_stride, const float* dh_last, void* dq, void* dk,
                  void* dv, float* dlog_decay, void* dbeta, float* dh0, void* workspace,
                  size_t workspace_bytes, void* stream) {
  const DeltaSizes s{batch, seqlen, nheads, nkheads, kdim, vdim, cu_seqlens != nullptr};
  int st = check_sizes(s, io_dtype);
  if (st != SSM_OK) return st;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (batch == 0) return SSM_OK;
  if (nheads == 0) {  // keys without value heads: sums over none
    if (nkheads == 0 || seqlen == 0) return SSM_OK;
    if (nkheads > kMaxHeads) return SSM_ERR_UNSUPPORTED;
    if (!dq || !dk || !all_aligned(dq, dk) || !aligned(cu_seqlens, 4) || !outputs_apart({dq, dk}, {q, k, cu_seqlens}))
      return SSM_ERR_INVALID_ARG;
    const int64_t row = nkheads * kdim * elem_bytes(io_dtype);
    hipError_t e = launch_zero_tokens(dq, row, s.tokens(), cu_seqlens, batch, hs);
    if (e == hipSuccess) e = launch_zero_tokens(dk, row, s.tokens(), cu_seqlens, batch, hs);
    return hip_status(e);
  }
  if (!all_aligned(h0, dh_last, dh0) || !outputs_apart({dh0}, {h0, dh_last}))
    return SSM_ERR_INVALID_ARG;
  if (seqlen == 0) {  // no token: the final state is the given one
    if (!dh0) return SSM_OK;
    return hip_status(launch_copy_state(dh_last, dh0, batch * nheads * s.state(), hs));
  }
  st = check_inputs(s, io_dtype, cu_seqlens, q, q_stride, k, k_stride, v, v_stride, log_decay, beta);
  if (st != SSM_OK) return st;
  if (!dy || !dq || !dk || !dv || !dlog_decay || !dbeta) return SSM_ERR_INVALID_ARG;
  if (!all_aligned(dy, dq, dk, dv, workspace) || !aligned(dlog_decay, 4) ||
      !aligned(dbeta, (unsigned)elem_bytes(io_dtype)))
    return SSM_ERR_INVALID_ARG;
  if ((st = check_stride(dy_stride, nheads, vdim, io_dtype)) != SSM_OK) return st;
  if (!outputs_apart({dq, dk, dv, dlog_decay, dbeta, dh0, workspace},
                     {q, k, v, log_decay, beta, h0, dy, dh_last, cu_seqlens}))
    return SSM_ERR_INVALID_ARG;
  const DeltaLayout l = layout_of(s, true, io_dtype);
  if (!workspace || workspace_bytes < l.total) return SSM_ERR_WORKSPACE;
  const bool bf16 = io_dtype == SSM_DTYPE_BF16;
  DeltaArgs a = delta_args(s, cu_seqlens, q, q_stride, k, k_stride, v, v_stride, log_decay, beta,
                           scale, h0, l, workspace, true, io_dtype);
  a.dy = {dy, dy_stride, 1};
  a.ds_last = dh_last;
  a.dq = dq, a.dk = dk, a.dv = dv;
  a.dlog_decay = dlog_decay;
  a.dbeta = dbeta;
  a.ds0 = dh0;
  hipError_t e = launch_delta_table(a, hs);
  if (e == hipSuccess) e = launch_delta_prep(a, bf16, hs);
  if (e == hipSuccess) e = launch_walk(a, bf16, hs);
  if (e == hipSuccess) e = launch_delta_grads(a, bf16, hs);
  return hip_status(e);
}

int ssm_delta_step(int64_t batch, int64_t nslots, const int32_t* slots, int64_t nheads,
                   int64_t nkheads, int64_t kdim, int64_t vdim, int io_dtype, float* h,
                   const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                   int64_t v_stride, const float* log_decay, const void* beta, float scale, void* o,
                   void* stream) {
  const DeltaSizes s{batch, 1, nheads, nkheads, kdim, vdim, false};
  int st = check_sizes(s, io_dtype);
  if (st != SSM_OK) return st;
  if (nslots < 0 || (!slots && nslots < batch)) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || nheads == 0) return SSM_OK;
  if (!h || !q || !k || !v || !log_decay || !beta || !o) return SSM_ERR_INVALID_ARG;
  if (!all_aligned(h, q, k, v, o) || !aligned(slots, 4) || !aligned(log_decay, 4) ||
      !aligned(beta, (unsigned)elem_bytes(io_dtype)))
    return SSM_ERR_INVALID_ARG;
  if ((st = check_free_stride(q_stride, nkheads, kdim, io_dtype)) != SSM_OK ||
      (st = check_free_stride(k_stride, nkheads, kdim, io_dtype)) != SSM_OK ||
      (st = check_free_stride(v_stride, nheads, vdim, io_dtype)) != SSM_OK)
    return st;
  if (!outputs_apart({h, o}, {q, k, v, log_decay, beta, slots})) return SSM_ERR_INVALID_ARG;
  DeltaStepArgs a{};
  const int rep = (int)(nheads / nkheads);
  a.h = h;
  a.slots = slots;
  a.q = {q, q_stride, rep};
  a.k = {k, k_stride, rep};
  a.v = {v, v_stride, 1};
  a.log_decay = log_decay;
  a.beta = beta;
  a.scale = scale;
  a.o = o;
  a.batch = batch;
  a.nslots = nslots;
  a.heads = (int)nheads;
  a.kd = (int)kdim;
  a.vd = (int)vdim;
  return hip_status(
      launch_delta_step(a, io_dtype == SSM_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Rows of a norm: any alignment of whole elements, any distance that holds a row.
int check_norm(int64_t rows, int64_t dim, int io_dtype, float eps) {
  if (rows < 0 || dim <= 0 || !valid_dtype(io_dtype) || !(eps >= 0.0f)) return SSM_ERR_INVALID_ARG;
  if (dim > kMaxNormDim || rows > kMaxFreeStride / dim) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}
int check_rows(const void* p, int64_t stride, int64_t rows, int64_t dim, int io_dtype) {
  if (!p || !aligned(p, (unsigned)elem_bytes(io_dtype)) || stride < dim) return SSM_ERR_INVALID_ARG;
  return stride > kMaxFreeStride / rows ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

}  // namespace

extern "C" {

int ssm_layer_norm_fwd(int64_t rows, int64_t dim, int io_dtype, const void* x, int64_t x_stride,
                       const float* weight, const float* bias, float eps, void* y, void* stream) {
  int st = check_norm(rows, dim, io_dtype, eps);
  if (st != SSM_OK) return st;
  if (rows == 0) return SSM_OK;
  if ((st = check_rows(x, x_stride, rows, dim, io_dtype)) != SSM_OK ||
      (st = check_rows(y, dim, rows, dim, io_dtype)) != SSM_OK)
    return st;
  if (!aligned(weight, 4) || !aligned(bias, 4) || !outputs_apart({y}, {x, weight, bias}))
    return SSM_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.w = weight;
  a.b = bias;
  a.out = y;
  a.rows = rows;
  a.dim = (int)dim;
  a.eps = eps;
  return hip_status(
      launch_norm_fwd(a, io_dtype == SSM_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

int64_t ssm_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int io_dtype) {
  if (check_norm(rows, dim, io_dtype, 0.0f) != SSM_OK) return -1;
  if (rows == 0) return 0;
  return (int64_t)norm_bwd_blocks(rows, (int)dim, io_dtype == SSM_DTYPE_BF16) * 2 * dim * 4;
}

int ssm_layer_norm_bwd(int64_t rows, int64_t dim, int io_dtype, const void* x, int64_t x_stride,
                       const float* weight, float eps, const void* dy, int64_t dy_stride, void* dx,
                       float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                       void* stream) {
  int st = check_norm(rows, dim, io_dtype, eps);
  if (st != SSM_OK) return st;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (!aligned(weight, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(workspace))
    return SSM_ERR_INVALID_ARG;
  if (rows == 0) {  // sums of nothing
    if ((dweight && dweight == dbias) || !outputs_apart({dweight, dbias}, {weight}))
      return SSM_ERR_INVALID_ARG;
    hipError_t e = hipSuccess;
    if (dweight) e = launch_copy_state(nullptr, dweight, dim, hs);
    if (e == hipSuccess && dbias) e = launch_copy_state(nullptr, dbias, dim, hs);
    return hip_status(e);
  }
  if ((st = check_rows(x, x_stride, rows, dim, io_dtype)) != SSM_OK ||
      (st = check_rows(dy, dy_stride, rows, dim, io_dtype)) != SSM_OK ||
      (st = check_rows(dx, dim, rows, dim, io_dtype)) != SSM_OK)
    return st;
  if (!outputs_apart({dx, dweight, dbias, workspace}, {x, weight, dy})) return SSM_ERR_INVALID_ARG;
  NormArgs a{};
  if (dweight || dbias) {
    const int64_t need = ssm_layer_norm_bwd_workspace_bytes(rows, dim, io_dtype);
    if (!workspace || workspace_bytes < (size_t)need) return SSM_ERR_WORKSPACE;
    a.part = static_cast<float*>(workspace);
  }
  a.x = x;
  a.dy = dy;
  a.x_stride = x_stride;
  a.dy_stride = dy_stride;
  a.w = weight;
  a.out = dx;
  a.dw = dweight;
  a.db = dbias;
  a.rows = rows;
  a.dim = (int)dim;
  a.eps = eps;
  return hip_status(launch_norm_bwd(a, io_dtype == SSM_DTYPE_BF16, hs));
}

}  // extern "C"
