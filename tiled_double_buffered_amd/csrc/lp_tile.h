// The product kernel that takes every case: any alignment, any leading dimension, any K,
// all operand orders.  64 x 64 tiles, four waves of 32 x 32, one LDS slot that registers
// prefetch for.  The larger products with 16-byte aligned rows go to the kernel of
// lp_pipe.h; this one is for the rest, and for products of few tiles.
#pragma once

#include "lp_common.h"

namespace gemmlp {

// Up to 16 bytes of a row from p; `n` elements of T are inside the row, the others read zero.
template <class T>
__device__ __forceinline__ int4v load_group(const typename T::type* p, int n) {
  constexpr int PER = 16 / T::BYTES;
  int4v v = {0, 0, 0, 0};
  if (n >= PER) {
    __builtin_memcpy(&v, p, 16);
  } else if (n > 0) {
    typename T::type e[PER] = {};
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < n) e[i] = p[i];
    __builtin_memcpy(&v, e, 16);
  }
  return v;
}

// One operand's part of a K step: 64 rows of 128 bytes in LDS, k contiguous, padded to 144
// bytes a row (16 rows then start at 16 different 16-byte groups of the banks).  KC: k is
// contiguous in memory too; otherwise the rows are, and the 16-byte groups that cross the
// rows are spread over them on the way into LDS.
constexpr int kTileRowStride = 144;
template <class T, bool KC>
struct TileOperand {
  static constexpr int PER = 16 / T::BYTES;
  static constexpr int KS = kRowBytes / T::BYTES;    // k in a step
  static constexpr int GROUPS = 64 * 8 / 256;        // 16-byte groups a thread moves
  static constexpr int CROSS = 64 / PER;             // groups across the 64 rows (!KC)
  int4v v[GROUPS];

  __device__ __forceinline__ void load(const typename T::type* base, int64_t ld, int r0,
                                       int r_end, int k0, int k_end, int tid) {
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const int g = tid + i * 256;
      if constexpr (KC) {
        const int r = r0 + g / 8, k = k0 + (g % 8) * PER;
        v[i] = load_group<T>(base + (int64_t)r * ld + k, r < r_end ? k_end - k : 0);
      } else {
        const int k = k0 + g / CROSS, r = r0 + (g % CROSS) * PER;
        v[i] = load_group<T>(base + (int64_t)k * ld + r, k < k_end ? r_end - r : 0);
      }
    }
  }
  __device__ __forceinline__ void store(char* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const int g = tid + i * 256;
      if constexpr (KC) {
        *(int4v*)(lds + (g / 8) * kTileRowStride + (g % 8) * 16) = v[i];
      } else {
        typename T::type e[PER];
        __builtin_memcpy(e, &v[i], 16);
        const int k = g / CROSS, r = (g % CROSS) * PER;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          *(typename T::type*)(lds + (r + j) * kTileRowStride + k * T::BYTES) = e[j];
      }
    }
  }
};

// AKC, BKC: k is contiguous in A (A[m][k], else A[k][m]) and in B (B[n][k], else B[k][n]).
// WGRAD: the group's rows are the contraction.
template <class T, bool AKC, bool BKC, bool WGRAD>
__global__ __launch_bounds__(256) void lp_tile_kernel(LpArgs p) {
  using E = typename T::type;
  __shared__ __align__(16) char lds[2 * 64 * kTileRowStride];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, lg = lane >> 4;

  const E* A = (const E*)p.A;
  const E* B = (const E*)p.B;
  int64_t c_base = 0;
  int m0, m_end, n0, e, k_end;
  if constexpr (WGRAD) {
    const int tiles_m = (p.M + 63) / 64, per = tiles_m * p.tiles_n;
    int tm, tn;
    wgrad_tile(blockIdx.x, per, tiles_m, p.tiles_n, e, tm, tn);
    const int lo = clamped_offset(p.offsets, e, p.rows);
    const int hi = clamped_offset(p.offsets, e + 1, p.rows);
    A += (int64_t)lo * p.lda;
    B += (int64_t)lo * p.ldb;
    k_end = max(hi - lo, 0);
    m0 = tm * 64;
    m_end = p.M;
    n0 = tn * 64;
    c_base = e * p.stride_c;
  } else {
    TileAt t;
    if (!find_tile<64, 0>(p, blockIdx.x, gridDim.x, t)) return;
    e = t.e;
    k_end = e < 0 ? 0 : p.K;
    if (e > 0) B += e * p.stride_b;
    m0 = t.row0;
    m_end = t.row_end;
    n0 = t.tn * 64;
  }

  float4v acc[2][2] = {};
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  TileOperand<T, AKC> ta;
  TileOperand<T, BKC> tb;
  char* la = lds;
  char* lb = lds + 64 * kTileRowStride;
  constexpr int KS = kRowBytes / T::BYTES;
  if (k_end > 0) {
    ta.load(A, p.lda, m0, m_end, 0, k_end, tid);
    tb.load(B, p.ldb, n0, p.N, 0, k_end, tid);
  }
  for (int k0 = 0, kt = 0; k0 < k_end; k0 += KS, ++kt) {
    __syncthreads();
    ta.store(la, tid);
    tb.store(lb, tid);
    __syncthreads();
    if (k0 + KS < k_end) {
      ta.load(A, p.lda, m0, m_end, k0 + KS, k_end, tid);
      tb.load(B, p.ldb, n0, p.N, k0 + KS, k_end, tid);
    }
    int4v alo[2], ahi[2], blo[2], bhi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char* ra = la + (wm + 16 * i + l16) * kTileRowStride + lg * 16;
      const char* rb = lb + (wn + 16 * i + l16) * kTileRowStride + lg * 16;
      alo[i] = *(const int4v*)ra;
      ahi[i] = *(const int4v*)(ra + 64);
      blo[i] = *(const int4v*)rb;
      bhi[i] = *(const int4v*)(rb + 64);
    }
    if constexpr (T::BYTES == 1) {
      // one K step is one block of scales: scale the step's sums, then add
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = min(m0 + wm + 16 * i + l16, m_end - 1);
        const float sa = p.SA[(int64_t)m * p.ldsa + kt];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4v z = {0.0f, 0.0f, 0.0f, 0.0f};
          const float4v d = mma_step<T>(blo[j], bhi[j], alo[i], ahi[i], z);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int n = min(n0 + wn + 16 * j + 4 * lg + r, p.N - 1);
            const float sb = p.SB[e * p.stride_sb + (int64_t)(n >> p.sb_shift) * p.ldsb + kt];
            acc[i][j][r] += d[r] * (sa * sb);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = mma_step<T>(blo[j], bhi[j], alo[i], ahi[i], acc[i][j]);
    }
  }

  const int cb = type_bytes(p.c_type);
  const bool vec = (((uintptr_t)p.C | (uintptr_t)(p.ldc * cb) | (uintptr_t)(c_base * cb)) &
                    (uintptr_t)(4 * cb - 1)) == 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = m0 + wm + 16 * i + l16;
    if (m >= m_end) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + wn + 16 * j + 4 * lg;
      store4(p.C, c_base + (int64_t)m * p.ldc + n, p.N - n, vec, p.c_type, acc[i][j]);
    }
  }
}

}  // namespace gemmlp
