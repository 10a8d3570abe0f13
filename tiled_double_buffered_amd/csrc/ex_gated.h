// The gated unit h = silu(g) u, silu(g) = g s(g), s(g) = 1 / (1 + exp(-g)), with g and u kept for
// its backward pass in 8 bits (or not kept: the backward pass then reads the input), and 8-bit
// values turned back into numbers.
//   dg = dh u s (1 + g (1 - s)),  du = dh g s
// s and 1 - s both come from exp(-|g|), so that neither is a difference of near numbers and the
// exponential never overflows.  For g < 0 s = c^3 r, c = exp(-|g| / 3) and r = 1 / (1 + c^3), and its
// three factors meet g, u and dh one by one: c is a normal number down to g = -262, where h is 0 for
// every u (and dg below 2^-113 for every u and dh), whereas exp(-|g|) is one only down to -87.
//
// Bound by memory: everything is read once and written once.  16 lanes hold a block of 128 columns,
// eight each, so that a block's scale needs four rotations.  16384 x 2048 in bf16, kept in 8 bits: 48
// us for 268 MB forward (5.6 TB/s, a part of it from the caches; 67 with the loads of gate and up
// behind a branch each), 42 us for as many backward; from its input 36 and 54; 16384 x 4096 values from 8 bits to bf16 38 us
// for 203 MB.
#pragma once

#include "ex_common.h"
#include "lp_quantize.h"

namespace gemmlp {

struct GatedArgs {
  const void* X;
  void* H;
  uint8_t* Q;        // the values kept: gate's N columns, then up's
  float* S;          // their scales: gate's blocks, then up's
  const void* DH;
  void* DX;
  int64_t ldx, ldh, ldq, lds, lddh, lddx;
  int rows, N;
};

// s(g) = c^3 r and 1 - s(g) = rest; c = 1 for g >= 0.  FP32 results keep the exponential's and the
// quotient's full precision; 16-bit ones, rounded at 2^-9 or 2^-12, take the instructions' (2^-22) for
// a third of the time.
struct Gate {
  float c, r, rest;
};
template <class T>
__device__ __forceinline__ Gate gate_of(float g) {
  float c, r;
  if constexpr (T::BYTES == 4) {
    c = expf(-(1.0f / 3.0f) * fabsf(g));
    r = 1.0f / (1.0f + c * c * c);
  } else {
    c = __builtin_amdgcn_exp2f(-0.480898347f * fabsf(g));  // log2 e / 3
    r = __builtin_amdgcn_rcpf(1.0f + c * c * c);
  }
  return g >= 0 ? Gate{1.0f, r, c * c * c * r} : Gate{c, r, r};
}

__device__ __forceinline__ void from_fp8x8(uint2 q, float scale, float* v) {
  typedef float float2v __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int w = (int)(i ? q.y : q.x);
    const float2v a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
    const float2v b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    v[4 * i] = a[0] * scale;
    v[4 * i + 1] = a[1] * scale;
    v[4 * i + 2] = b[0] * scale;
    v[4 * i + 3] = b[1] * scale;
  }
}
__device__ __forceinline__ uint2 load_bytes8(const uint8_t* p, int n) {
  typedef uint32_t group __attribute__((ext_vector_type(2), aligned(1)));
  if (n >= 8) {
    const group g = *(const group*)p;
    return make_uint2(g[0], g[1]);
  }
  uint2 q = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) (i < 4 ? q.x : q.y) |= (uint32_t)p[i] << (8 * (i & 3));
  return q;
}

// load8 of several rows, all of them under way together: one branch for all, as the loads before a
// branch have to arrive at it.
template <class T, class P, class V>
__device__ __forceinline__ void load8_each(int n, P p, V v) {
  load8<T>(p, n, v);
}
template <class T, class P, class V, class... More>
__device__ __forceinline__ void load8_each(int n, P p, V v, More... more) {
  load8<T>(p, n, v);
  load8_each<T>(n, more...);
}
template <class T, class... PV>
__device__ __forceinline__ void load8s(int n, PV... pv) {
  if (n >= 8) load8_each<T>(8, pv...);
  else load8_each<T>(n, pv...);
}

// Eight 8-bit values times their scale, as numbers of T's range: finite products past it become its
// largest number (T's own largest can round up to such a product).
template <class T>
__device__ __forceinline__ void dequantized(uint2 q, float scale, float* v) {
  constexpr float most = T::CODE == GEMM_LP_F16    ? 65504.0f
                         : T::CODE == GEMM_LP_BF16 ? 3.3895313892515355e38f
                                                   : 3.4028234663852886e38f;
  from_fp8x8(q, scale, v);
  if (fabsf(scale) < __builtin_inff()) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(v[i]) > most) v[i] = copysignf(most, v[i]);
  }
}

// Which row, block and first column a thread has; false past the end (for whole 16 lanes).
__device__ __forceinline__ bool block_at(int rows, int cols, int& row, int& block, int& c) {
  const int kb = (cols + kBlock - 1) / kBlock;
  const int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (unit >= (int64_t)rows * kb) return false;
  row = (int)(unit / kb);
  block = (int)(unit - (int64_t)row * kb);
  c = block * kBlock + (threadIdx.x & 15) * 8;
  return true;
}

__device__ __forceinline__ int block_exponent(const float* v) {
  float top = max_over_16(top_of<8, true>(v, 1));
  if (top == __builtin_inff()) top = max_over_16(top_of<8, false>(v, 1));
  return scale_exponent(top);
}

template <class T, bool KEEP>
__global__ __launch_bounds__(256) void ex_gated_kernel(GatedArgs p) {
  int row, block, c;
  if (!block_at(p.rows, p.N, row, block, c)) return;
  const int n = p.N - c;
  const typename T::type* x = (const typename T::type*)p.X + row * p.ldx + c;
  float g[8], u[8], h[8];
  load8s<T>(n, x, g, x + p.N, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Gate t = gate_of<T>(g[i]);
    h[i] = g[i] * t.c * t.r * (u[i] * t.c) * t.c;
  }
  store_row<8, T::CODE>(p.H, row * p.ldh + c, n, T::CODE, h);
  if constexpr (KEEP) {
    const int eg = block_exponent(g), eu = block_exponent(u);
    uint8_t* q = p.Q + row * p.ldq + c;
    store_bytes8(q, n, to_fp8x8(g, 1, power_of_two(eg)));
    store_bytes8(q + p.N, n, to_fp8x8(u, 1, power_of_two(eu)));
    if ((threadIdx.x & 15) == 0) {
      float* s = p.S + row * p.lds + block;
      s[0] = power_of_two(eg);
      s[(p.N + kBlock - 1) / kBlock] = power_of_two(eu);
    }
  }
}

template <class T, bool KEEP>
__global__ __launch_bounds__(256) void ex_gated_grad_kernel(GatedArgs p) {
  int row, block, c;
  if (!block_at(p.rows, p.N, row, block, c)) return;
  const int n = p.N - c;
  float g[8], u[8], dh[8];
  const typename T::type* d = (const typename T::type*)p.DH + row * p.lddh + c;
  if constexpr (KEEP) {
    const uint8_t* q = p.Q + row * p.ldq + c;
    const float* s = p.S + row * p.lds + block;
    const float sg = s[0], su = s[(p.N + kBlock - 1) / kBlock];
    uint2 qg, qu;
    if (n >= 8) {
      qg = load_bytes8(q, 8), qu = load_bytes8(q + p.N, 8);
      load8<T>(d, 8, dh);
    } else {
      qg = load_bytes8(q, n), qu = load_bytes8(q + p.N, n);
      load8<T>(d, n, dh);
    }
    dequantized<T>(qg, sg, g);
    dequantized<T>(qu, su, u);
  } else {
    const typename T::type* x = (const typename T::type*)p.X + row * p.ldx + c;
    load8s<T>(n, x, g, x + p.N, u, d, dh);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Gate t = gate_of<T>(g[i]);
    const float slope = t.c * (t.r * (1.0f + g[i] * t.rest)), silu = g[i] * t.c * t.r;
    g[i] = slope * dh[i] * (u[i] * t.c) * t.c;
    u[i] = silu * (dh[i] * t.c) * t.c;
  }
  store_row<8, T::CODE>(p.DX, row * p.lddx + c, n, T::CODE, g);
  store_row<8, T::CODE>(p.DX, row * p.lddx + p.N + c, n, T::CODE, u);
}

struct DequantArgs {
  const uint8_t* Q;
  const float* S;
  void* Y;
  int64_t ldq, lds, ldy;
  int rows, cols, shift;  // shift: log2 of the rows of a block
};

template <class T>
__global__ __launch_bounds__(256) void ex_dequantize_kernel(DequantArgs p) {
  int row, block, c;
  if (!block_at(p.rows, p.cols, row, block, c)) return;
  const int n = p.cols - c;
  const float scale = p.S[(int64_t)(row >> p.shift) * p.lds + block];
  float v[8];
  dequantized<T>(load_bytes8(p.Q + row * p.ldq + c, n), scale, v);
  store_row<8, T::CODE>(p.Y, row * p.ldy + c, n, T::CODE, v);
}

}  // namespace gemmlp
