// Host: the checks of arguments and the launch that the low-precision and expert entry points share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "lp_common.h"

namespace gemmlp {

constexpr int64_t kMaxDim = 2147483647LL - 1024;  // keeps tile-end arithmetic in int32
constexpr int64_t kMaxExtent = (int64_t)1 << 61;   // bytes one operand may span

// Byte range [lo, hi) of `count` blocks of rows x cols values of `bytes` bytes, row stride ld
// and block stride `stride` (elements).  False where it passes kMaxExtent or wraps.
struct Range {
  uintptr_t lo = 0, hi = 0;
};
static inline bool byte_range(const void* p, int64_t count, int64_t stride, int64_t rows, int64_t cols,
                       int64_t ld, int64_t bytes, Range* r) {
  int64_t e, s;
  if (__builtin_mul_overflow(rows - 1, ld, &e) || __builtin_add_overflow(e, cols, &e) ||
      __builtin_mul_overflow(count - 1, stride, &s) || __builtin_add_overflow(e, s, &e) ||
      __builtin_mul_overflow(e, bytes, &e) || e > kMaxExtent)
    return false;
  r->lo = (uintptr_t)p;
  return !__builtin_add_overflow(r->lo, (uintptr_t)e, &r->hi);
}
static inline bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// Outputs against each other and against inputs; unused ranges are empty and overlap nothing.
template <int OUTS, int INS>
static inline bool any_overlap(const Range (&out)[OUTS], const Range (&in)[INS]) {
  for (int i = 0; i < OUTS; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}
static inline bool row_range(const void* p, int64_t count, int64_t bytes, Range* r) {
  return byte_range(p, 1, 0, 1, count, count, bytes, r);
}

static inline bool known_type(int t) { return t == GEMM_LP_BF16 || t == GEMM_LP_F16 || t == GEMM_LP_F32; }
static inline bool misaligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) != 0; }
static inline int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }
static inline int64_t at_least_1(int64_t n) { return n > 1 ? n : 1; }

static inline int launch(const void* fn, dim3 grid, int threads, void* args, void* stream) {
  void* list[] = {args};
  const hipError_t err =
      hipLaunchKernel(fn, grid, dim3((unsigned)threads), list, 0, (hipStream_t)stream);
  if (err != hipSuccess) {
    gemmf32::set_last_hip_error((int)err);
    return GEMMF32_ERR_HIP;
  }
  return GEMMF32_OK;
}

}  // namespace gemmlp
