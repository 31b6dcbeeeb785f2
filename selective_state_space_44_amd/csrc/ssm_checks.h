// ssm_checks.h -- argument checks on the host that the entry points of the linear
// attention, the delta rule and the norms share.
// Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "ssm.h"

namespace ssm {

constexpr int64_t kMaxHeads = 1 << 20;
// Elements between tokens: where a chunk of 64 tokens of one operand is addressed
// with 32-bit byte offsets, and where every token has a 64-bit address (no tensor
// on this card is larger).
constexpr int64_t kMaxStride = (int64_t)1 << 22;
constexpr int64_t kMaxFreeStride = (int64_t)1 << 38;
constexpr int64_t kMaxBlocks = INT32_MAX;

inline bool valid_dtype(int t) { return t == SSM_DTYPE_F32 || t == SSM_DTYPE_BF16; }
inline int64_t elem_bytes(int t) { return t == SSM_DTYPE_BF16 ? 2 : 4; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }
inline bool aligned(const void* p, unsigned to = 16) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}
template <typename... P> bool all_aligned(P... p) { return (aligned(p) && ...); }

typedef std::initializer_list<const void*> Ptrs;

// No output (a non-null one) is an input or another output.
inline bool outputs_apart(Ptrs outs, Ptrs ins) {
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
inline int check_stride(int64_t stride, int64_t heads, int64_t dim, int io_dtype,
                        int64_t most = kMaxStride) {
  if (stride < heads * dim || (stride * elem_bytes(io_dtype)) % 16 != 0) return SSM_ERR_INVALID_ARG;
  return stride > most ? SSM_ERR_UNSUPPORTED : SSM_OK;
}
inline int check_free_stride(int64_t stride, int64_t heads, int64_t dim, int io_dtype) {
  return check_stride(stride, heads, dim, io_dtype, kMaxFreeStride);
}

inline size_t align_up(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace ssm
