// Quantization to 8-bit floating point with one power-of-two scale for each block.
//
// The scale of a block whose largest finite magnitude is a is 2^e, e the smallest integer
// >= -126 with a <= 448 * 2^e.  With a = 1.m * 2^(E - 127) (E and m the fields of the FP32
// number) and 448 = 1.75 * 2^8, e = E - 135 where 1.m <= 1.75 and one more above, so the
// exponent field and one comparison give it; the division by 2^e is exact but for values that
// become subnormal, far below half of the format's smallest step, and the one rounding is the
// conversion instruction's, to nearest with ties to even.
//
// Bound by memory: every value is read once, whatever is asked for, and 8 bits of it written once
// or twice.  8192 x 8192 in bf16 with its transpose takes 64 to 66 us for 273 MB, 4.1 to 4.3 of
// the 5.1 TB/s that a large copy reaches; 4096 x 4096 in 128 x 128 blocks with its transpose
// 16.5 to 19; 16 x 4096 takes 2.5 us, a launch and one reading's latency.  A
// thread holds 8 x 8 values, so that the scales by rows and by columns and both orders of the
// result come from one reading (92 us with a check of every value for Inf, which the maxima now
// make unnecessary but for one test a workgroup).
#pragma once

#include <type_traits>

#include "lp_common.h"

namespace gemmlp {

// EXP: the scales as bytes e + 127, one for each row of Q and block of columns (the rows of a
// block all get its exponent), block by block: S[block * lds + row].  Otherwise as FP32 numbers,
// one for each block: S[row block * lds + block].
struct QuantArgs {
  const void* X;
  uint8_t* Q;
  void* S;
  uint8_t* QT;
  void* ST;
  int64_t ldx, ldq, lds, ldqt, ldst;
  int rows, cols;
};

__device__ __forceinline__ int scale_exponent(float top) {  // top: finite, not negative
  const uint32_t bits = __builtin_bit_cast(uint32_t, top);
  const int e = (int)(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -126);
}
__device__ __forceinline__ float power_of_two(int e) {
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}
// Eight values over 2^e as 8-bit numbers: the conversion divides by the power of two, rounds to
// nearest even, and turns Inf and NaN into NaN.
__device__ __forceinline__ uint2 to_fp8x8(const float* v, int step, float scale) {
  typedef short short2v __attribute__((ext_vector_type(2)));
  short2v lo = {0, 0}, hi = {0, 0};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[0], v[step], scale, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[2 * step], v[3 * step], scale, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[4 * step], v[5 * step], scale, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[6 * step], v[7 * step], scale, true);
  return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

// Eight neighbouring values of a row, the first `n` of them inside it.
template <class T>
__device__ __forceinline__ void load8(const typename T::type* p, int n, float* v) {
  typedef typename T::type E;
  typedef E group __attribute__((ext_vector_type(8), aligned(sizeof(E))));
  if (n >= 8) {
    const group e = *(const group*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? (float)p[i] : 0.0f;
  }
}
__device__ __forceinline__ void store_bytes8(uint8_t* p, int n, uint2 q) {
  typedef uint32_t group __attribute__((ext_vector_type(2), aligned(1)));
  if (n >= 8) {
    *(group*)p = group{q.x, q.y};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

// Maxima over lanes: over each 16 by rotations on the vector unit, and over the four 16s of a
// wave.
__device__ __forceinline__ float max_over_16(float m) {
  auto turn = [&](auto ctrl) {
    const int v = __builtin_bit_cast(int, m);
    m = fmaxf(m, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                               v, v, decltype(ctrl)::value, 0xf, 0xf, false)));
  };
  turn(std::integral_constant<int, 0x121>{});  // row_ror:1
  turn(std::integral_constant<int, 0x122>{});
  turn(std::integral_constant<int, 0x124>{});
  turn(std::integral_constant<int, 0x128>{});
  return m;
}
__device__ __forceinline__ float max_over_rows(float m) {
  m = fmaxf(m, __shfl_xor(m, 16));
  return fmaxf(m, __shfl_xor(m, 32));
}

// The largest finite magnitude of values v[0], v[step], ...; NO_INF: it is known that none is
// Inf (a maximum passes over NaN by itself).
template <int N, bool NO_INF>
__device__ __forceinline__ float top_of(const float* v, int step) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float a = fabsf(v[i * step]);
    m = fmaxf(m, NO_INF || a < __builtin_inff() ? a : 0.0f);
  }
  return m;
}

template <bool EXP>
__device__ __forceinline__ void put_scale(void* S, int64_t ld, int row, int block, int e) {
  if constexpr (EXP) ((uint8_t*)S)[block * ld + row] = (uint8_t)(e + 127);
  else ((float*)S)[row * ld + block] = power_of_two(e);
}

// 1 x 128 blocks, no transpose: 16 lanes a block, 16 blocks a workgroup.
template <class T, bool EXP>
__global__ __launch_bounds__(256) void lp_quantize_rows_kernel(QuantArgs p) {
  const int kb = (p.cols + kBlock - 1) / kBlock;
  const int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (unit >= (int64_t)p.rows * kb) return;  // whole groups of 16 lanes
  const int row = (int)(unit / kb), b = (int)(unit - (int64_t)row * kb);
  const int c = b * kBlock + (threadIdx.x & 15) * 8;
  float v[8];
  load8<T>((const typename T::type*)p.X + row * p.ldx + c, p.cols - c, v);
  float top = max_over_16(top_of<8, true>(v, 1));
  if (top == __builtin_inff()) top = max_over_16(top_of<8, false>(v, 1));
  const int e = scale_exponent(top);
  store_bytes8(p.Q + row * p.ldq + c, p.cols - c, to_fp8x8(v, 1, power_of_two(e)));
  if ((threadIdx.x & 15) == 0) put_scale<EXP>(p.S, p.lds, row, b, e);
}

// A 128 x 128 tile whose values the threads hold (lp_quantize_tile_kernel).
constexpr int kTurnStride = kBlock + 16;
template <int ROWS, bool EXP, bool NO_INF>
__device__ __forceinline__ void quantize_tile(const QuantArgs& p, const float (&v)[8][8],
                                              float (&part)[4][kBlock], uint8_t* turn, int bm,
                                              int bk) {
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, wave = tid >> 6;
  const int r0 = bm * kBlock, c0 = bk * kBlock;
  const int c = c0 + tx * 8;
  if constexpr (ROWS == 1) {
    if (p.Q != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + ty * 8 + i;
        const int e = scale_exponent(max_over_16(top_of<8, NO_INF>(v[i], 1)));
        if (r < p.rows) {
          store_bytes8(p.Q + r * p.ldq + c, p.cols - c, to_fp8x8(v[i], 1, power_of_two(e)));
          if (tx == 0) put_scale<EXP>(p.S, p.lds, r, bk, e);
        }
      }
    }
    if (p.QT == nullptr) return;
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = max_over_rows(top_of<8, NO_INF>(&v[0][j], 8));
    if ((tid & 63) < 16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) part[wave][tx * 8 + j] = m[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = tx * 8 + j;
      const int e =
          scale_exponent(fmaxf(fmaxf(part[0][k], part[1][k]), fmaxf(part[2][k], part[3][k])));
      *(uint2*)(turn + k * kTurnStride + ty * 8) = to_fp8x8(&v[0][j], 8, power_of_two(e));
      if (ty == 0 && c0 + k < p.cols) put_scale<EXP>(p.ST, p.ldst, c0 + k, bm, e);
    }
  } else {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, top_of<8, NO_INF>(v[i], 1));
    m = max_over_rows(max_over_16(m));
    if ((tid & 63) == 0) part[0][wave] = m;
    __syncthreads();
    const int e =
        scale_exponent(fmaxf(fmaxf(part[0][0], part[0][1]), fmaxf(part[0][2], part[0][3])));
    const float scale = power_of_two(e);
    if (p.Q != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + ty * 8 + i;
        if (r < p.rows) store_bytes8(p.Q + r * p.ldq + c, p.cols - c, to_fp8x8(v[i], 1, scale));
      }
      if constexpr (EXP) {
        if (tid < kBlock && r0 + tid < p.rows) put_scale<EXP>(p.S, p.lds, r0 + tid, bk, e);
      } else {
        if (tid == 0) put_scale<EXP>(p.S, p.lds, bm, bk, e);
      }
    }
    if (p.QT == nullptr) return;
    if constexpr (EXP) {
      if (tid < kBlock && c0 + tid < p.cols) put_scale<EXP>(p.ST, p.ldst, c0 + tid, bm, e);
    } else {
      if (tid == 0) put_scale<EXP>(p.ST, p.ldst, bk, bm, e);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *(uint2*)(turn + (tx * 8 + j) * kTurnStride + ty * 8) = to_fp8x8(&v[0][j], 8, scale);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = i * 32 + (tid >> 3), r = r0 + (tid & 7) * 16;
    if (c0 + k >= p.cols) continue;
    const uint4 q = *(const uint4*)(turn + k * kTurnStride + (tid & 7) * 16);
    uint8_t* to = p.QT + (c0 + k) * p.ldqt + r;
    if (r + 16 <= p.rows) {
      typedef uint32_t group __attribute__((ext_vector_type(4), aligned(1)));
      *(group*)to = group{q.x, q.y, q.z, q.w};
    } else {
      store_bytes8(to, p.rows - r, make_uint2(q.x, q.y));
      store_bytes8(to + 8, p.rows - r - 8, make_uint2(q.z, q.w));
    }
  }
}

// 128 x 128 tiles: thread (ty, tx) of 16 x 16 holds rows 8 ty .. + 7, columns 8 tx .. + 7, so
// that X is read once whatever is asked for.  ROWS: rows of a block (1 or 128).
template <class T, int ROWS, bool EXP>
__global__ __launch_bounds__(256) void lp_quantize_tile_kernel(QuantArgs p) {
  __shared__ float part[4][kBlock];
  __shared__ __align__(16) uint8_t turn[kBlock * kTurnStride];
  // (one axis of workgroups: the others end at 65535 of them)
  const int tid = threadIdx.x, kb = (p.cols + kBlock - 1) / kBlock;
  const int bm = blockIdx.x / kb, bk = blockIdx.x - bm * kb;
  const int r0 = bm * kBlock + (tid >> 4) * 8, c = bk * kBlock + (tid & 15) * 8;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load8<T>((const typename T::type*)p.X + (r0 + i) * p.ldx + c,
             r0 + i < p.rows ? p.cols - c : 0, v[i]);
  // one maximum decides for the workgroup whether Inf has to be looked for
  float any = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) any = fmaxf(any, top_of<8, true>(v[i], 1));
  if (__syncthreads_or(any == __builtin_inff()))
    quantize_tile<ROWS, EXP, false>(p, v, part, turn, bm, bk);
  else
    quantize_tile<ROWS, EXP, true>(p, v, part, turn, bm, bk);
}

}  // namespace gemmlp
