// Quantization to 8-bit floating point with one power-of-two scale for each block.
//
// The scale of a block whose largest finite magnitude is a is 2^e, e the smallest integer
// >= -126 with a <= 448 * 2^e.  With a = 1.m * 2^(E - 127) (E and m the fields of the FP32
// number) and 448 = 1.75 * 2^8, e = E - 135 where 1.m <= 1.75 and one more above, so the
// exponent field and one comparison give it; the division by 2^e is exact but for values that
// become subnormal, far below half of the format's smallest step, and the one rounding is the
// conversion instruction's, to nearest with ties to even.
#pragma once

#include "lp_common.h"

namespace gemmlp {

struct QuantArgs {
  const void* X;
  uint8_t* Q;
  float* S;
  uint8_t* QT;
  float* ST;
  int64_t ldx, ldq, lds, ldqt, ldst;
  int rows, cols;
};

__device__ __forceinline__ uint32_t finite_bits(float x) {  // |x| as bits, 0 for Inf and NaN
  const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int e = (int)(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -126);
}
__device__ __forceinline__ float power_of_two(int e) {
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}
// Two values as 8-bit numbers in the low or high half of `old`.
template <bool HIGH>
__device__ __forceinline__ int to_fp8(float a, float b, float inv, int old) {
  a = finite_bits(a) || a == 0.0f ? a * inv : __builtin_nanf("");
  b = finite_bits(b) || b == 0.0f ? b * inv : __builtin_nanf("");
  return __builtin_amdgcn_cvt_pk_fp8_f32(a, b, old, HIGH);
}
__device__ __forceinline__ uint2 to_fp8x8(const float* v, int step, float inv) {
  int lo = 0, hi = 0;
  lo = to_fp8<false>(v[0], v[step], inv, lo);
  lo = to_fp8<true>(v[2 * step], v[3 * step], inv, lo);
  hi = to_fp8<false>(v[4 * step], v[5 * step], inv, hi);
  hi = to_fp8<true>(v[6 * step], v[7 * step], inv, hi);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Eight neighbouring values of a row, the first `n` of them inside it.
template <class T>
__device__ __forceinline__ void load8(const typename T::type* p, int n, float* v) {
  typename T::type e[8];
  if (n >= 8) {
    __builtin_memcpy(e, p, sizeof(e));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : (typename T::type)0.0f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
}
__device__ __forceinline__ void store_bytes8(uint8_t* p, int n, uint2 q) {
  if (n >= 8) {
    __builtin_memcpy(p, &q, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

__device__ __forceinline__ uint32_t max_over_16(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 16; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  return m;
}

// 1 x 128 blocks, no transpose: 16 lanes a block, 16 blocks a workgroup.
template <class T>
__global__ __launch_bounds__(256) void lp_quantize_rows_kernel(QuantArgs p) {
  const int kb = (p.cols + kBlock - 1) / kBlock;
  const int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (unit >= (int64_t)p.rows * kb) return;  // whole groups of 16 lanes
  const int row = (int)(unit / kb), b = (int)(unit - (int64_t)row * kb);
  const int c = b * kBlock + (threadIdx.x & 15) * 8;
  float v[8];
  load8<T>((const typename T::type*)p.X + row * p.ldx + c, p.cols - c, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, finite_bits(v[i]));
  const int e = scale_exponent(max_over_16(m));
  store_bytes8(p.Q + row * p.ldq + c, p.cols - c, to_fp8x8(v, 1, power_of_two(-e)));
  if ((threadIdx.x & 15) == 0) p.S[row * p.lds + b] = power_of_two(e);
}

// 128 x 128 tiles: thread (ty, tx) of 16 x 16 holds rows 8 ty .. + 7, columns 8 tx .. + 7, so
// that X is read once whatever is asked for.  ROWS: rows of a block (1 or 128).
template <class T, int ROWS>
__global__ __launch_bounds__(256) void lp_quantize_tile_kernel(QuantArgs p) {
  __shared__ uint32_t part[4][kBlock];
  constexpr int kStride = kBlock + 16;
  __shared__ __align__(16) uint8_t turn[kBlock * kStride];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, wave = tid >> 6;
  const int r0 = blockIdx.y * kBlock, c0 = blockIdx.x * kBlock;
  const int c = c0 + tx * 8;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + ty * 8 + i;
    load8<T>((const typename T::type*)p.X + r * p.ldx + c, r < p.rows ? p.cols - c : 0, v[i]);
  }
  if constexpr (ROWS == 1) {
    if (p.Q != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + ty * 8 + i;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, finite_bits(v[i][j]));
        const int e = scale_exponent(max_over_16(m));
        if (r < p.rows) {
          store_bytes8(p.Q + r * p.ldq + c, p.cols - c, to_fp8x8(v[i], 1, power_of_two(-e)));
          if (tx == 0) p.S[r * p.lds + blockIdx.x] = power_of_two(e);
        }
      }
    }
    if (p.QT == nullptr) return;
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[j] = max(m[j], finite_bits(v[i][j]));
      m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 16));
      m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 32));
    }
    if ((tid & 63) < 16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) part[wave][tx * 8 + j] = m[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = tx * 8 + j;
      const int e = scale_exponent(max(max(part[0][k], part[1][k]), max(part[2][k], part[3][k])));
      *(uint2*)(turn + k * kStride + ty * 8) = to_fp8x8(&v[0][j], 8, power_of_two(-e));
      if (ty == 0 && c0 + k < p.cols) p.ST[(c0 + k) * p.ldst + blockIdx.y] = power_of_two(e);
    }
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, finite_bits(v[i][j]));
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if ((tid & 63) == 0) part[0][wave] = m;
    __syncthreads();
    const int e = scale_exponent(max(max(part[0][0], part[0][1]), max(part[0][2], part[0][3])));
    const float inv = power_of_two(-e);
    if (p.Q != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + ty * 8 + i;
        if (r < p.rows) store_bytes8(p.Q + r * p.ldq + c, p.cols - c, to_fp8x8(v[i], 1, inv));
      }
      if (tid == 0) p.S[blockIdx.y * p.lds + blockIdx.x] = power_of_two(e);
    }
    if (p.QT == nullptr) return;
    if (tid == 0) p.ST[blockIdx.x * p.ldst + blockIdx.y] = power_of_two(e);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *(uint2*)(turn + (tx * 8 + j) * kStride + ty * 8) = to_fp8x8(&v[0][j], 8, inv);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = i * 32 + (tid >> 3), r = r0 + (tid & 7) * 16;
    if (c0 + k >= p.cols) continue;
    const uint4 q = *(const uint4*)(turn + k * kStride + (tid & 7) * 16);
    uint8_t* to = p.QT + (c0 + k) * p.ldqt + r;
    if (r + 16 <= p.rows) {
      __builtin_memcpy(to, &q, 16);
    } else {
      store_bytes8(to, p.rows - r, make_uint2(q.x, q.y));
      store_bytes8(to + 8, p.rows - r - 8, make_uint2(q.z, q.w));
    }
  }
}

}  // namespace gemmlp
