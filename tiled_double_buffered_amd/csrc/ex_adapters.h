// Adapters of low rank, each for a group of rows: out = y + s_e (x A_e^T) B_e with A_e rank x K and
// B_e rank x N, and their gradients.  With u = s x A^T and v = s dout B^T,
//   out = y + u B,  dx = v A,  dA = v^T x,  dB = u^T dout,
// so that three kernels serve all of it: `down` (u, v: the contraction is the wide axis), `up`
// (out, dx: the contraction is the rank) and `grad` (dA, dB: it is the group's rows).  As A and B
// both have the wide axis contiguous, every kernel reads all of its operands in whole lines.
//
// u and v stay in FP32 between the kernels.  `down` multiplies 16-bit values by the 16-bit matrix
// instruction (exact products, FP32 sums); `up` and `grad`, one of whose operands is u or v, take
// the FP32 instruction, whose operands hold one k a lane: neither operand needs turning.
#pragma once

#include "ex_common.h"

namespace gemmlp {

struct AdapterArgs {
  LpArgs p;  // A: the rows, B: the adapters, C: the result; M: rank, N: the wide axis; offsets, E
  const int64_t* order;
  const float* scale;
  const void* Y;
  float* U;
  float* part;     // grad: [split of rows][E][rank][N], where there are several
  int64_t ldy;
  int splits;      // of U
  int k_chunk;     // down: columns of a split
  int row_splits;  // grad
};

__device__ __forceinline__ int64_t row_at(const AdapterArgs& a, int place) {
  const int64_t r = a.order[place];
  return min(max(r, (int64_t)0), (int64_t)a.p.rows - 1);
}

// COUNT neighbouring values as they are, zeros past the first n.
template <class T, int COUNT>
__device__ __forceinline__ auto load_raw(const typename T::type* p, int n) {
  typedef typename T::type E;
  typedef E group __attribute__((ext_vector_type(COUNT)));
  typedef E any __attribute__((ext_vector_type(COUNT), aligned(sizeof(E))));
  group v;
  if (n >= COUNT) {
    v = *(const any*)p;
  } else {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) v[i] = i < n ? p[i] : (E)0.0f;
  }
  return v;
}

__device__ __forceinline__ float4v mma16(bf168v a, bf168v b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float4v mma16(half8v a, half8v b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float4v mma32(float a, float b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// u of 16 places and one split of K.  Four waves take turns at steps of K; the instruction's rows
// are the rank, its columns the places.  RF: fragments of 16 of the rank.
constexpr int kDownThreads = 256;
template <class T, int RF>
__global__ __launch_bounds__(kDownThreads) void ex_adapters_down_kernel(AdapterArgs a) {
  constexpr int PER = 16 / T::BYTES;      // values of one load
  constexpr int STEP = 4 * 2 * PER;       // of K: two loads of each of the four lane groups
  constexpr int LD = RF * 16 + 4;
  __shared__ float red[4][16][LD];
  const LpArgs& p = a.p;
  TileAt t;
  if (!find_tile<16, 0>(p, blockIdx.x, gridDim.x, t) || t.e < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const typename T::type* x =
      (const typename T::type*)p.A + row_at(a, min(t.row0 + l16, t.row_end - 1)) * p.lda;
  const typename T::type* w = (const typename T::type*)p.B + t.e * p.stride_b;
  const typename T::type* wr[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) wr[f] = w + min(16 * f + l16, p.M - 1) * p.ldb;
  float4v acc[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) acc[f] = float4v{0, 0, 0, 0};
  const int first = (int)min((int64_t)t.tn * a.k_chunk, (int64_t)p.K);
  const int end = first + min(a.k_chunk, p.K - first);
  for (int k0 = first + wave * STEP; k0 < end; k0 += 4 * STEP) {
    const int k = k0 + g * 2 * PER;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kk = k + h * PER, n = end - kk;
      const auto xv = load_raw<T, PER>(x + kk, n);
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        const auto wv = load_raw<T, PER>(wr[f] + kk, n);
        if constexpr (T::BYTES == 4) {
#pragma unroll
          for (int j = 0; j < PER; ++j) acc[f] = mma32(wv[j], xv[j], acc[f]);
        } else {
          acc[f] = mma16(wv, xv, acc[f]);
        }
      }
    }
  }
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[wave][l16][16 * f + 4 * g + q] = acc[f][q];
  __syncthreads();
  const float s = a.scale != nullptr ? a.scale[t.e] : 1.0f;
  float* u = a.U + (int64_t)t.tn * p.rows * p.M;
  for (int i = tid; i < 16 * RF * 16; i += kDownThreads) {
    const int row = i / (RF * 16), r = i % (RF * 16);
    if (t.row0 + row < t.row_end && r < p.M)
      u[(int64_t)(t.row0 + row) * p.M + r] =
          s * ((red[0][row][r] + red[1][row][r]) + (red[2][row][r] + red[3][row][r]));
  }
}

// u at (place, r): the splits' sum.
__device__ __forceinline__ float u_at(const AdapterArgs& a, int place, int r) {
  const float* u = a.U + (int64_t)place * a.p.M + r;
  float v = *u;
  for (int s = 1; s < a.splits; ++s) v += u[(int64_t)s * a.p.rows * a.p.M];
  return v;
}

// 16 places x 512 columns, a wave 128 of them.  The instruction's rows are columns of the result:
// fragment j takes column 8 i + j for its row i, so that a lane loads eight neighbours of B at
// once and ends with 32 neighbouring columns of one place.
constexpr int kUpThreads = 256, kWaveCols = 128, kUpCols = 4 * kWaveCols;
template <class T>
__global__ __launch_bounds__(kUpThreads) void ex_adapters_up_kernel(AdapterArgs a) {
  const LpArgs& p = a.p;
  TileAt t;
  if (!find_tile<16, 0>(p, blockIdx.x, gridDim.x, t)) return;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int n0 = t.tn * kUpCols + (threadIdx.x >> 6) * kWaveCols;
  if (n0 >= p.N) return;
  const int place = min(t.row0 + l16, t.row_end - 1);
  const int64_t row = row_at(a, place);
  float4v acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = float4v{0, 0, 0, 0};
  if (t.e >= 0) {
    const typename T::type* b = (const typename T::type*)p.B + t.e * p.stride_b + n0 + 8 * l16;
    const int n = p.N - n0 - 8 * l16;
    for (int r0 = 0; r0 < p.M; r0 += 4) {
      const int r = r0 + g;
      const float u = r < p.M ? u_at(a, place, r) : 0.0f;
      float w[8];
      load_row<T, 8>(b + r * p.ldb, r < p.M ? n : 0, 0.0f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = mma32(w[j], u, acc[j]);
    }
  }
  if (t.row0 + l16 >= t.row_end) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int c = n0 + 32 * g + 8 * q, n = p.N - c;
    float v[8];
    if (a.Y != nullptr) {
      load_row<T, 8>((const typename T::type*)a.Y + row * a.ldy + c, n, 0.0f, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += acc[j][q];
    store_row<8, T::CODE>(p.C, row * p.ldc + c, n, T::CODE, v);
  }
}

// 128 columns of RF * 16 rows of one expert's gradient.  The waves take turns at 16 of the group's
// places and add up through LDS; row_splits workgroups share a group's places.
template <int RF>
struct GradShape {
  static constexpr int WAVES = RF <= 2 ? 8 : 4;
};
template <class T, int RF>
__global__ __launch_bounds__(GradShape<RF>::WAVES * 64) void ex_adapters_grad_kernel(AdapterArgs a) {
  constexpr int WAVES = GradShape<RF>::WAVES, N = RF * 8 * 4;
  __shared__ float red[WAVES / 2][N][64];
  const LpArgs& p = a.p;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  // workgroups: columns, then row splits, then blocks of the rank, then experts
  const int rb = (p.M + RF * 16 - 1) / (RF * 16);
  int id = blockIdx.x;
  const int n0 = id % p.tiles_n * kWaveCols;
  id /= p.tiles_n;
  const int split = id % a.row_splits;
  id /= a.row_splits;
  const int r0 = id % rb * (RF * 16), e = id / rb;
  const int lo = clamped_offset(p.offsets, e, p.rows);
  const int len = max(clamped_offset(p.offsets, e + 1, p.rows) - lo, 0);
  const int first = lo + (int)((int64_t)len * split / a.row_splits);
  const int end = lo + (int)((int64_t)len * (split + 1) / a.row_splits);
  float4v acc[RF][8];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[f][j] = float4v{0, 0, 0, 0};
  const typename T::type* x = (const typename T::type*)p.A + n0 + 8 * l16;
  const int n = p.N - n0 - 8 * l16;
  for (int i0 = first + wave * 16; i0 < end; i0 += WAVES * 16) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int place = i0 + 4 * s + g;
      const bool in = place < end;
      float v[8], u[RF];
      load_row<T, 8>(x + row_at(a, in ? place : first) * p.lda, in ? n : 0, 0.0f, v);
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        const int r = r0 + 16 * f + l16;
        u[f] = in && r < p.M ? u_at(a, place, r) : 0.0f;
      }
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[f][j] = mma32(v[j], u[f], acc[f][j]);
    }
  }
  for (int d = WAVES / 2; d > 0; d /= 2) {
    if (wave >= d && wave < 2 * d) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave - d][i][lane] = acc[i / 32][i / 4 % 8][i % 4];
    }
    __syncthreads();
    if (wave < d) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i / 32][i / 4 % 8][i % 4] += red[wave][i][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int f = 0; f < RF; ++f) {
    const int r = r0 + 16 * f + l16;
    if (r >= p.M) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = n0 + 32 * g + 8 * q;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[f][j][q];
      if (a.row_splits > 1) {
        const int64_t at = (((int64_t)split * p.E + e) * p.M + r) * p.N + c;
        store_row<8, GEMM_LP_F32>(a.part, at, p.N - c, GEMM_LP_F32, v);
      } else {
        store_row<8, T::CODE>(p.C, e * p.stride_c + r * p.ldc + c, p.N - c, T::CODE, v);
      }
    }
  }
}

// The sum of the row splits' parts; a thread has eight columns.
template <class T>
__global__ __launch_bounds__(256) void ex_adapters_sum_kernel(AdapterArgs a) {
  const LpArgs& p = a.p;
  const int per = (p.N + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.E * p.M * per) return;
  const int64_t row = i / per;  // e * rank + r
  const int c = (int)(i - row * per) * 8, n = p.N - c;
  float v[8] = {};
  for (int s = 0; s < a.row_splits; ++s) {
    float w[8];
    load_row<F32, 8>(a.part + ((int64_t)s * p.E * p.M + row) * p.N + c, n, 0.0f, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += w[j];
  }
  const int e = (int)(row / p.M), r = (int)(row - (int64_t)e * p.M);
  store_row<8, T::CODE>(p.C, e * p.stride_c + r * p.ldc + c, n, T::CODE, v);
}

}  // namespace gemmlp
