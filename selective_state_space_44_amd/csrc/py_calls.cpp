// py_calls.cpp -- the binding's quick way into the calls that are made once per
// token and layer (CPython module _calls).
//
// A call made from Python spends more on looking at its tensors and on
// marshalling than on launching (a decode step's rotation: 12.2 us, 2.6 of them
// the launch; here 5.6).  Each function below takes the address of the library's
// entry point and the tensors as the binding's function got them.  It checks that
// everything is as the entry point needs it, allocates the outputs and the
// workspace and calls on the current stream of the tensors' device.  It answers
// None when anything is not as it should be (the binding's own checks then find
// out what, and raise), the status when the call fails, else the outputs.  It
// keeps nothing between calls.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>

#include <cstdint>
#include <vector>

#include "ssm.h"

namespace {

using at::Tensor;

// What a function returns early with: not as it should be.
struct Unusual {};

void need(bool ok) {
  if (!ok) throw Unusual{};
}

const Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  need(!(v == -1 && PyErr_Occurred()));
  return v;
}
template <typename F> F function(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  need(p != nullptr);
  return reinterpret_cast<F>(p);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  need(!(v == -1.0 && PyErr_Occurred()));
  return (float)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  need(v >= 0);
  return v != 0;
}

// What the operands of a call share.
struct Kind {
  at::ScalarType type;
  at::Device device;
  int code;
  void* stream() const { return c10::hip::getCurrentHIPStream(device.index()).stream(); }
};
Kind kind_of(const Tensor& t) {
  const at::ScalarType type = t.scalar_type();
  need(t.is_cuda() && (type == at::kFloat || type == at::kBFloat16));
  return {type, t.device(), type == at::kFloat ? SSM_DTYPE_F32 : SSM_DTYPE_BF16};
}

// Address of a contiguous tensor of these sizes.
template <typename T = float>
T* whole(PyObject* o, at::IntArrayRef sizes, at::ScalarType type, const Kind& kind) {
  const Tensor& t = tensor(o);
  need(t.scalar_type() == type && t.device() == kind.device && t.sizes() == sizes &&
       t.is_contiguous());
  return static_cast<T*>(t.data_ptr());
}
template <typename T = float>
T* optional(PyObject* o, at::IntArrayRef sizes, at::ScalarType type, const Kind& kind) {
  return o == Py_None ? nullptr : whole<T>(o, sizes, type, kind);
}

// Elements between the evenly spaced tokens of a [..., tokens, heads, dim] tensor
// whose last two dimensions are contiguous.
int64_t token_stride(const Tensor& t) {
  const at::IntArrayRef n = t.sizes(), s = t.strides();
  const size_t d = n.size();
  const int64_t heads = n[d - 2], dim = n[d - 1];
  if (t.is_contiguous()) return heads * dim;
  need((s[d - 1] == 1 || dim == 1) && (s[d - 2] == dim || heads == 1));
  if (d == 3 || n[0] == 1) return n[d - 3] > 1 ? s[d - 3] : heads * dim;
  if (n[1] == 1) return s[0];
  need(s[0] == n[1] * s[1]);
  return s[1];
}

struct Strided {
  void* p;
  int64_t stride;
};
Strided strided(const Tensor& t, at::IntArrayRef sizes, const Kind& kind) {
  need(t.scalar_type() == kind.type && t.device() == kind.device && t.sizes() == sizes);
  return {t.data_ptr(), token_stride(t)};
}

// `shape` with its last two sizes replaced.
std::vector<int64_t> with(at::IntArrayRef shape, int64_t heads, int64_t dim) {
  std::vector<int64_t> v(shape.begin(), shape.end());
  v[v.size() - 2] = heads;
  v[v.size() - 1] = dim;
  return v;
}

Tensor fresh(const Tensor& like, at::IntArrayRef sizes) { return at::empty(sizes, like.options()); }
Tensor fresh(const Tensor& like, at::IntArrayRef sizes, at::ScalarType type) {
  return at::empty(sizes, like.options().dtype(type));
}
Tensor workspace(const Tensor& like, int64_t bytes) {
  need(bytes >= 0);
  return bytes ? fresh(like, {bytes}, at::kByte) : Tensor();
}
template <typename T = void> T* data(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}
size_t bytes_of(const Tensor& t) { return t.defined() ? (size_t)t.numel() : 0; }

// Runs a call without the interpreter's lock (a full queue makes it wait).
template <typename F> int unlocked(F&& f) {
  PyThreadState* s = PyEval_SaveThread();
  const int status = f();
  PyEval_RestoreThread(s);
  return status;
}

PyObject* wrapped(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
// The outputs, or the status of a call that failed.
PyObject* answer(int status, std::initializer_list<const Tensor*> outputs) {
  if (status != SSM_OK) return PyLong_FromLong(status);
  PyObject* r = PyTuple_New((Py_ssize_t)outputs.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* t : outputs) {
    PyObject* o = wrapped(*t);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// No exception leaves a function: whatever is raised on the way is left to the
// binding's own checks.
template <typename F> PyObject* guarded(Py_ssize_t n, Py_ssize_t expected, F&& f) {
  if (n == expected) {
    try {
      return f();
    } catch (...) {
      PyErr_Clear();
    }
  }
  Py_RETURN_NONE;
}

// --- head norm with rotation -----------------------------------------------
struct RotateCall {
  const Tensor &q, &k;
  Kind kind;
  int64_t tokens, seqlen, hq, hk, dim, half = 0, npos = 0;
  Strided qs, ks;
  const float *cos = nullptr, *sin = nullptr, *qw, *kw;
  const int64_t* positions;

  // a: q, k, cos, sin, positions, q_weight, k_weight
  explicit RotateCall(PyObject* const* a) : q(tensor(a[0])), k(tensor(a[1])), kind(kind_of(q)) {
    const at::IntArrayRef n = q.sizes();
    const size_t d = n.size();
    need((d == 3 || d == 4) && (size_t)k.dim() == d);
    dim = n[d - 1], hq = n[d - 2], seqlen = n[d - 3], hk = k.size(d - 2);
    tokens = d == 3 ? seqlen : n[0] * seqlen;
    qs = strided(q, n, kind);
    ks = strided(k, with(n, hk, dim), kind);
    if (a[2] != Py_None || a[3] != Py_None) {
      const Tensor& c = tensor(a[2]);
      need(c.dim() == 2);
      npos = c.size(0), half = c.size(1);
      cos = whole(a[2], c.sizes(), at::kFloat, kind);
      sin = whole(a[3], c.sizes(), at::kFloat, kind);
    }
    positions = optional<int64_t>(a[4], n.slice(0, d - 2), at::kLong, kind);
    need(half == 0 || positions || seqlen <= npos);
    qw = optional(a[5], {dim}, at::kFloat, kind);
    kw = optional(a[6], {dim}, at::kFloat, kind);
  }
};

// (function, q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved)
//  -> q, k
PyObject* rotate_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_qk_norm_rotate_fwd)>(a[0]);
    const RotateCall c(a + 1);
    const float eps = real(a[8]);
    const int interleaved = truth(a[9]);
    void* stream = c.kind.stream();
    const Tensor qo = fresh(c.q, c.q.sizes()), ko = fresh(c.k, c.k.sizes());
    const int st = unlocked([&] {
      return fn(c.tokens, c.seqlen, c.hq, c.hk, c.dim, 2 * c.half, interleaved, c.kind.code, c.qs.p,
                c.qs.stride, c.ks.p, c.ks.stride, c.cos, c.sin, c.npos, c.positions, c.qw, c.kw,
                eps, data(qo), data(ko), stream);
    });
    return answer(st, {&qo, &ko});
  });
}

// (function, workspace function, q, k, cos, sin, positions, q_weight, k_weight, eps,
//  interleaved, dq_out, dk_out, need_dweight) -> dq, dk, dq_weight, dk_weight
PyObject* rotate_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_qk_norm_rotate_bwd)>(a[0]);
    const auto size = function<decltype(&ssm_qk_norm_rotate_bwd_workspace_bytes)>(a[1]);
    const RotateCall c(a + 2);
    const float eps = real(a[9]);
    const int interleaved = truth(a[10]);
    const Strided dqo = strided(tensor(a[11]), c.q.sizes(), c.kind);
    const Strided dko = strided(tensor(a[12]), c.k.sizes(), c.kind);
    const bool weights = truth(a[13]);
    void* stream = c.kind.stream();
    const Tensor dq = fresh(c.q, c.q.sizes()), dk = fresh(c.k, c.k.sizes());
    Tensor dqw, dkw, ws;
    if (weights && c.qw) dqw = fresh(c.q, {c.dim}, at::kFloat);
    if (weights && c.kw) dkw = fresh(c.q, {c.dim}, at::kFloat);
    if (dqw.defined() || dkw.defined()) ws = workspace(c.q, size(c.tokens, c.hq, c.hk, c.dim));
    const int st = unlocked([&] {
      return fn(c.tokens, c.seqlen, c.hq, c.hk, c.dim, 2 * c.half, interleaved, c.kind.code, c.qs.p,
                c.qs.stride, c.ks.p, c.ks.stride, c.cos, c.sin, c.npos, c.positions, c.qw, c.kw,
                eps, dqo.p, dqo.stride, dko.p, dko.stride, data(dq), data(dk), data<float>(dqw),
                data<float>(dkw), data(ws), bytes_of(ws), stream);
    });
    return answer(st, {&dq, &dk, &dqw, &dkw});
  });
}

// --- linear attention --------------------------------------------------------
struct AttnCall {
  const Tensor &q, &k, &v;
  Kind kind;
  int64_t batch, seqlen, heads, kv, kdim, vdim;
  const int32_t* cu = nullptr;
  Strided qs, ks, vs;
  const float *decay, *h0;

  // a: q, k, v, log_decay, h0, cu_seqlens
  explicit AttnCall(PyObject* const* a)
      : q(tensor(a[0])), k(tensor(a[1])), v(tensor(a[2])), kind(kind_of(q)) {
    const at::IntArrayRef n = q.sizes();
    const size_t d = n.size();
    need(d == (a[5] == Py_None ? 4u : 3u) && (size_t)k.dim() == d && (size_t)v.dim() == d);
    heads = n[d - 2], kdim = n[d - 1], kv = k.size(d - 2), vdim = v.size(d - 1);
    if (a[5] == Py_None) {
      batch = n[0], seqlen = n[1];
    } else {
      const Tensor& c = tensor(a[5]);
      need(c.dim() == 1 && c.numel() >= 1);
      cu = whole<int32_t>(a[5], c.sizes(), at::kInt, kind);
      batch = c.numel() - 1, seqlen = n[0];
      need(batch > 0 || seqlen == 0);
    }
    need(heads == 0 || (kv > 0 && heads % kv == 0));
    qs = strided(q, n, kind);
    ks = strided(k, with(n, kv, kdim), kind);
    vs = strided(v, with(n, kv, vdim), kind);
    decay = whole(a[3], {heads}, at::kFloat, kind);
    h0 = optional(a[4], {batch, heads, vdim, kdim}, at::kFloat, kind);
  }
  Tensor state() const { return fresh(q, {batch, heads, vdim, kdim}, at::kFloat); }
};

// (function, workspace function, q, k, v, log_decay, h0, cu_seqlens, scale,
//  return_last_state, nsplit) -> o, h_last
PyObject* linattn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_linattn_fwd)>(a[0]);
    const auto size = function<decltype(&ssm_linattn_fwd_workspace_bytes)>(a[1]);
    const AttnCall c(a + 2);
    const float scale = real(a[8]);
    const bool last = truth(a[9]);
    const int nsplit = (int)integer(a[10]);
    void* stream = c.kind.stream();
    const Tensor o = fresh(c.q, with(c.q.sizes(), c.heads, c.vdim));
    const Tensor h = last ? c.state() : Tensor();
    const Tensor ws = workspace(c.q, size(c.batch, c.seqlen, c.cu != nullptr, c.heads, c.kv, c.kdim,
                                          c.vdim, c.kind.code, nsplit));
    const int st = unlocked([&] {
      return fn(c.batch, c.seqlen, c.cu, c.heads, c.kv, c.kdim, c.vdim, c.kind.code, c.qs.p,
                c.qs.stride, c.ks.p, c.ks.stride, c.vs.p, c.vs.stride, c.decay, scale, c.h0,
                data(o), data<float>(h), nsplit, data(ws), bytes_of(ws), stream);
    });
    return answer(st, {&o, &h});
  });
}

// (function, workspace function, q, k, v, log_decay, h0, cu_seqlens, scale, dy, dh_last,
//  need_dlog_decay, need_dh0, nsplit) -> dq, dk, dv, dlog_decay, dh0
PyObject* linattn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_linattn_bwd)>(a[0]);
    const auto size = function<decltype(&ssm_linattn_bwd_workspace_bytes)>(a[1]);
    const AttnCall c(a + 2);
    const float scale = real(a[8]);
    const Strided dy = strided(tensor(a[9]), with(c.q.sizes(), c.heads, c.vdim), c.kind);
    const float* dh =
        optional(a[10], {c.batch, c.heads, c.vdim, c.kdim}, at::kFloat, c.kind);
    const bool decay = truth(a[11]), state = truth(a[12]);
    const int nsplit = (int)integer(a[13]);
    void* stream = c.kind.stream();
    const Tensor dq = fresh(c.q, c.q.sizes()), dk = fresh(c.k, c.k.sizes()),
                 dv = fresh(c.v, c.v.sizes());
    const Tensor dg = decay ? fresh(c.q, {c.heads}, at::kFloat) : Tensor();
    const Tensor dh0 = state ? c.state() : Tensor();
    const Tensor ws = workspace(c.q, size(c.batch, c.seqlen, c.cu != nullptr, c.heads, c.kv, c.kdim,
                                          c.vdim, c.kind.code, decay, nsplit));
    const int st = unlocked([&] {
      return fn(c.batch, c.seqlen, c.cu, c.heads, c.kv, c.kdim, c.vdim, c.kind.code, c.qs.p,
                c.qs.stride, c.ks.p, c.ks.stride, c.vs.p, c.vs.stride, c.decay, scale, c.h0, dy.p,
                dy.stride, dh, data(dq), data(dk), data(dv), data<float>(dg), data<float>(dh0),
                nsplit, data(ws), bytes_of(ws), stream);
    });
    return answer(st, {&dq, &dk, &dv, &dg, &dh0});
  });
}

// (function, h, q, k, v, log_decay, scale, slots) -> (o,)
PyObject* linattn_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_linattn_step)>(a[0]);
    const Tensor &h = tensor(a[1]), &q = tensor(a[2]), &k = tensor(a[3]), &v = tensor(a[4]);
    need(h.dim() == 4 && q.dim() == 3 && k.dim() == 3);
    const Kind kind = kind_of(q);
    const int64_t nslots = h.size(0), heads = h.size(1), vdim = h.size(2), kdim = h.size(3);
    const int64_t batch = q.size(0), kv = k.size(1);
    need(heads == 0 || (kv > 0 && heads % kv == 0));
    float* state = whole(a[1], h.sizes(), at::kFloat, kind);
    const Strided qs = strided(q, {batch, heads, kdim}, kind), ks = strided(k, {batch, kv, kdim}, kind),
                  vs = strided(v, {batch, kv, vdim}, kind);
    const float* decay = whole(a[5], {heads}, at::kFloat, kind);
    const float scale = real(a[6]);
    const int32_t* slots = optional<int32_t>(a[7], {batch}, at::kInt, kind);
    need(slots || nslots >= batch);
    void* stream = kind.stream();
    const Tensor o = fresh(q, {batch, heads, vdim});
    const int st = unlocked([&] {
      return fn(batch, nslots, slots, heads, kv, kdim, vdim, kind.code, state, qs.p, qs.stride, ks.p,
                ks.stride, vs.p, vs.stride, decay, scale, data(o), stream);
    });
    // a state that is kept for a backward pass has changed
    if (st == SSM_OK && !h.is_inference()) h.unsafeGetTensorImpl()->bump_version();
    return answer(st, {&o});
  });
}

// --- gated delta rule ----------------------------------------------------------
struct DeltaCall {
  const Tensor &q, &k, &v;
  Kind kind;
  int64_t batch, seqlen, heads, kheads, kdim, vdim;
  const int32_t* cu = nullptr;
  Strided qs, ks, vs;
  const float *decay, *h0;
  const void* beta;
  std::vector<int64_t> gates;  // shape of log_decay and beta

  // a: q, k, v, log_decay, beta, h0, cu_seqlens
  explicit DeltaCall(PyObject* const* a)
      : q(tensor(a[0])), k(tensor(a[1])), v(tensor(a[2])), kind(kind_of(q)) {
    const at::IntArrayRef n = q.sizes();
    const size_t d = n.size();
    need(d == (a[6] == Py_None ? 4u : 3u) && (size_t)k.dim() == d && (size_t)v.dim() == d);
    kheads = n[d - 2], kdim = n[d - 1], heads = v.size(d - 2), vdim = v.size(d - 1);
    if (a[6] == Py_None) {
      batch = n[0], seqlen = n[1];
    } else {
      const Tensor& c = tensor(a[6]);
      need(c.dim() == 1 && c.numel() >= 1);
      cu = whole<int32_t>(a[6], c.sizes(), at::kInt, kind);
      batch = c.numel() - 1, seqlen = n[0];
      need(batch > 0 || seqlen == 0);
    }
    need(heads == 0 || (kheads > 0 && heads % kheads == 0));
    qs = strided(q, n, kind);
    ks = strided(k, n, kind);
    vs = strided(v, with(n, heads, vdim), kind);
    gates.assign(n.begin(), n.end() - 1);
    gates.back() = heads;
    decay = whole(a[3], gates, at::kFloat, kind);
    beta = whole<void>(a[4], gates, kind.type, kind);
    h0 = optional(a[5], {batch, heads, vdim, kdim}, at::kFloat, kind);
  }
  Tensor state() const { return fresh(q, {batch, heads, vdim, kdim}, at::kFloat); }
};

// (function, workspace function, q, k, v, log_decay, beta, h0, cu_seqlens, scale,
//  return_last_state) -> o, h_last
PyObject* delta_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_delta_fwd)>(a[0]);
    const auto size = function<decltype(&ssm_delta_fwd_workspace_bytes)>(a[1]);
    const DeltaCall c(a + 2);
    const float scale = real(a[9]);
    const bool last = truth(a[10]);
    void* stream = c.kind.stream();
    const Tensor o = fresh(c.v, c.v.sizes());
    const Tensor h = last ? c.state() : Tensor();
    const Tensor ws = workspace(c.q, size(c.batch, c.seqlen, c.cu != nullptr, c.heads, c.kheads,
                                          c.kdim, c.vdim, c.kind.code));
    const int st = unlocked([&] {
      return fn(c.batch, c.seqlen, c.cu, c.heads, c.kheads, c.kdim, c.vdim, c.kind.code, c.qs.p,
                c.qs.stride, c.ks.p, c.ks.stride, c.vs.p, c.vs.stride, c.decay, c.beta, scale, c.h0,
                data(o), data<float>(h), data(ws), bytes_of(ws), stream);
    });
    return answer(st, {&o, &h});
  });
}

// (function, workspace function, q, k, v, log_decay, beta, h0, cu_seqlens, scale, dy,
//  dh_last, need_dh0) -> dq, dk, dv, dlog_decay, dbeta, dh0
PyObject* delta_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_delta_bwd)>(a[0]);
    const auto size = function<decltype(&ssm_delta_bwd_workspace_bytes)>(a[1]);
    const DeltaCall c(a + 2);
    const float scale = real(a[9]);
    const Strided dy = strided(tensor(a[10]), c.v.sizes(), c.kind);
    const float* dh = optional(a[11], {c.batch, c.heads, c.vdim, c.kdim}, at::kFloat, c.kind);
    const bool state = truth(a[12]);
    void* stream = c.kind.stream();
    const Tensor dq = fresh(c.q, c.q.sizes()), dk = fresh(c.k, c.k.sizes()),
                 dv = fresh(c.v, c.v.sizes());
    const Tensor dg = fresh(c.q, c.gates, at::kFloat), db = fresh(c.q, c.gates);
    const Tensor dh0 = state ? c.state() : Tensor();
    const Tensor ws = workspace(c.q, size(c.batch, c.seqlen, c.cu != nullptr, c.heads, c.kheads,
                                          c.kdim, c.vdim, c.kind.code));
    const int st = unlocked([&] {
      return fn(c.batch, c.seqlen, c.cu, c.heads, c.kheads, c.kdim, c.vdim, c.kind.code, c.qs.p,
                c.qs.stride, c.ks.p, c.ks.stride, c.vs.p, c.vs.stride, c.decay, c.beta, scale, c.h0,
                dy.p, dy.stride, dh, data(dq), data(dk), data(dv), data<float>(dg), data(db),
                data<float>(dh0), data(ws), bytes_of(ws), stream);
    });
    return answer(st, {&dq, &dk, &dv, &dg, &db, &dh0});
  });
}

// (function, h, q, k, v, log_decay, beta, scale, slots) -> (o,)
PyObject* delta_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_delta_step)>(a[0]);
    const Tensor &h = tensor(a[1]), &q = tensor(a[2]), &k = tensor(a[3]), &v = tensor(a[4]);
    need(h.dim() == 4 && q.dim() == 3);
    const Kind kind = kind_of(q);
    const int64_t nslots = h.size(0), heads = h.size(1), vdim = h.size(2), kdim = h.size(3);
    const int64_t batch = q.size(0), kheads = q.size(1);
    need(heads == 0 || (kheads > 0 && heads % kheads == 0));
    float* state = whole(a[1], h.sizes(), at::kFloat, kind);
    const Strided qs = strided(q, {batch, kheads, kdim}, kind),
                  ks = strided(k, {batch, kheads, kdim}, kind),
                  vs = strided(v, {batch, heads, vdim}, kind);
    const float* decay = whole(a[5], {batch, heads}, at::kFloat, kind);
    const void* beta = whole<void>(a[6], {batch, heads}, kind.type, kind);
    const float scale = real(a[7]);
    const int32_t* slots = optional<int32_t>(a[8], {batch}, at::kInt, kind);
    need(slots || nslots >= batch);
    void* stream = kind.stream();
    const Tensor o = fresh(q, {batch, heads, vdim});
    const int st = unlocked([&] {
      return fn(batch, nslots, slots, heads, kheads, kdim, vdim, kind.code, state, qs.p, qs.stride,
                ks.p, ks.stride, vs.p, vs.stride, decay, beta, scale, data(o), stream);
    });
    // a state that is kept for a backward pass has changed
    if (st == SSM_OK && !h.is_inference()) h.unsafeGetTensorImpl()->bump_version();
    return answer(st, {&o});
  });
}

// --- layer norm ------------------------------------------------------------------
// Address of a [..., dim] tensor with contiguous, evenly spaced rows, and the
// elements between them.
Strided rows_of(const Tensor& t, at::IntArrayRef sizes, const Kind& kind) {
  need(t.scalar_type() == kind.type && t.device() == kind.device && t.sizes() == sizes);
  const int64_t d = (int64_t)sizes.size(), dim = sizes[d - 1];
  if (t.is_contiguous()) return {t.data_ptr(), dim};
  need(t.stride(d - 1) == 1 || dim == 1);
  int64_t step = -1, rows = 1;
  for (int64_t i = d - 2; i >= 0; --i) {
    if (sizes[i] == 1) continue;
    if (step < 0) step = t.stride(i);
    else need(t.stride(i) == rows * step);
    rows *= sizes[i];
  }
  return {t.data_ptr(), step < 0 ? dim : step};
}

// (function, x, weight, bias, eps) -> (y,)
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_layer_norm_fwd)>(a[0]);
    const Tensor& x = tensor(a[1]);
    const Kind kind = kind_of(x);
    need(x.dim() >= 1 && x.size(x.dim() - 1) > 0);
    const int64_t dim = x.size(x.dim() - 1), rows = x.numel() / dim;
    const Strided xs = rows_of(x, x.sizes(), kind);
    const float *w = optional(a[2], {dim}, at::kFloat, kind), *b = optional(a[3], {dim}, at::kFloat, kind);
    const float eps = real(a[4]);
    void* stream = kind.stream();
    const Tensor y = fresh(x, x.sizes());
    const int st = unlocked(
        [&] { return fn(rows, dim, kind.code, xs.p, xs.stride, w, b, eps, data(y), stream); });
    return answer(st, {&y});
  });
}

// (function, workspace function, x, weight, dy, eps, need_dweight, need_dbias)
//  -> dx, dweight, dbias
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const auto fn = function<decltype(&ssm_layer_norm_bwd)>(a[0]);
    const auto size = function<decltype(&ssm_layer_norm_bwd_workspace_bytes)>(a[1]);
    const Tensor& x = tensor(a[2]);
    const Kind kind = kind_of(x);
    need(x.dim() >= 1 && x.size(x.dim() - 1) > 0);
    const int64_t dim = x.size(x.dim() - 1), rows = x.numel() / dim;
    const Strided xs = rows_of(x, x.sizes(), kind), dy = rows_of(tensor(a[4]), x.sizes(), kind);
    const float* w = optional(a[3], {dim}, at::kFloat, kind);
    const float eps = real(a[5]);
    const bool dweight = truth(a[6]), dbias = truth(a[7]);
    void* stream = kind.stream();
    const Tensor dx = fresh(x, x.sizes());
    Tensor dw, db, ws;
    if (dweight) dw = fresh(x, {dim}, at::kFloat);
    if (dbias) db = fresh(x, {dim}, at::kFloat);
    if (dweight || dbias) ws = workspace(x, size(rows, dim, kind.code));
    const int st = unlocked([&] {
      return fn(rows, dim, kind.code, xs.p, xs.stride, w, eps, dy.p, dy.stride, data(dx),
                data<float>(dw), data<float>(db), data(ws), bytes_of(ws), stream);
    });
    return answer(st, {&dx, &dw, &db});
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(F), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<rotate_fwd>("rotate_fwd"),   method<rotate_bwd>("rotate_bwd"),
                         method<linattn_fwd>("linattn_fwd"), method<linattn_bwd>("linattn_bwd"),
                         method<linattn_step>("linattn_step"), method<delta_fwd>("delta_fwd"),
                         method<delta_bwd>("delta_bwd"),     method<delta_step>("delta_step"),
                         method<norm_fwd>("norm_fwd"),       method<norm_bwd>("norm_bwd"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
