// Shared parts of the low-precision and expert-grouped products: element types, the matrix
// instructions, kernel arguments, the search for a workgroup's tile in ragged groups of rows,
// and the epilogue's stores.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_lp.h"

namespace gemmlp {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int8v __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf168v __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;   // columns (along K) that share a scale
constexpr int kRowBytes = 128;  // bytes of one operand row in a K step, every type
constexpr int kXcds = 8, kCus = 256;

struct Bf16 {
  using type = __bf16;
  static constexpr int BYTES = 2;
  static constexpr int CODE = GEMM_LP_BF16;
};
struct F16 {
  using type = _Float16;
  static constexpr int BYTES = 2;
  static constexpr int CODE = GEMM_LP_F16;
};
struct F32 {
  using type = float;
  static constexpr int BYTES = 4;
  static constexpr int CODE = GEMM_LP_F32;
};
struct F8 {
  using type = uint8_t;
  static constexpr int BYTES = 1;
  static constexpr int CODE = -1;
};

static inline __host__ __device__ int type_bytes(int code) { return code == GEMM_LP_F32 ? 4 : 2; }

// Eight 8-bit values as halves.
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ half8v fp8x8_to_half(int w0, int w1) {
  const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false);
  const half2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true);
  const half2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false);
  const half2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true);
  return half8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The product of two 16-row operands of 8-bit values over one K step of 128.  Lane l holds of row
// l % 16 the two 16-byte groups lo and hi that its lane group l / 16 stands for; both operands
// use the same groups, so that the order of k inside the step does not matter.  D's row index
// comes from `a`, its column from `b`: lane l, register r hold row 4 (l / 16) + r, column l % 16.
// The values go through the 16-bit instruction, which every e4m3 number fits exactly and whose
// sums hold FP32's 24 bits below their largest product.  The 8-bit instructions (16x16x128 and
// 16x16x32 alike) hold 13 bits below the largest of each eight neighbouring products:
// 256 * 256 - 256 * 256 + 2 * 2 comes out as 0, and sums of values of all sizes are off by up to
// 2^-12.5 of their magnitudes (2^-15.4 in the mean square; the 16-bit one 2^-21.3 and 2^-24).
__device__ __forceinline__ float4v mma_fp8_step(int4v alo, int4v ahi, int4v blo, int4v bhi,
                                                float4v c) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int4v a = i ? ahi : alo, b = i ? bhi : blo;
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(fp8x8_to_half(a[0], a[1]),
                                               fp8x8_to_half(b[0], b[1]), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(fp8x8_to_half(a[2], a[3]),
                                               fp8x8_to_half(b[2], b[3]), c, 0, 0, 0);
  }
  return c;
}

// Arguments of every product kernel.  Row products: C rows m0.. of group e from A's rows and
// B_e.  Weight gradients: the group's rows are the contraction, M x N the size of one C_e.
struct LpArgs {
  const void* A;
  const void* B;
  void* C;
  const float* SA;
  const float* SB;
  const int32_t* offsets;  // NULL: one group of all rows
  int64_t lda, ldb, ldc;   // elements
  int64_t stride_b;        // elements from one expert's B to the next's (row products)
  int64_t stride_c;        // elements from one expert's C to the next's (weight gradients)
  int64_t ldsa, ldsb, stride_sb;
  int rows;                // rows of A: M of a row product, the contraction of a gradient
  int M, N, K;             // row products: M = rows; gradients: K = rows
  int E;
  int tiles_n;
  int sb_shift;            // log2 of the rows of B that share a scale: 7 or 0
  int c_type;
};

// One expert's rows, from the offsets: clamped to [0, rows], empty where they decrease.
__device__ __forceinline__ int clamped_offset(const int32_t* off, int i, int rows) {
  return min(max(off[i], 0), rows);
}

struct TileAt {
  int e;         // expert (0 where there are no offsets); -1: rows of no expert
  int row0;      // first row of the tile
  int row_end;   // end of the group's rows
  int tn;        // tile column
  bool half;     // HALF rows or fewer
};

// Consecutive ids for the workgroups of one XCD: workgroup w runs on XCD w mod 8, and
// XCD x gets ids x q + min(x, r) .. of n = 8 q + r, a permutation of 0 .. n - 1.
__device__ __forceinline__ int xcd_order(int w, int n) {
  const int q = n / kXcds, r = n % kXcds, x = w % kXcds;
  return x * q + min(x, r) + w / kXcds;
}

// Tiles of one group are walked in bands of kBand tile rows, column by column, so that the
// workgroups of one XCD that run together share rows of A and of B in its L2 (8192^3 in
// bf16: 763 us in bands of 4, 763 of 6, 760 of 8, 784 of 16; in 8 bits 933, 930, 918, 950).
constexpr int kBand = 4;
__device__ __forceinline__ void band_order(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int band = id / (kBand * tiles_n);
  const int rest = id - band * kBand * tiles_n;
  const int h = min(kBand, tiles_m - band * kBand);
  tn = rest / h;
  tm = band * kBand + rest - tn * h;
}

// Weight gradients: workgroup wg computes tile (tm, tn) of expert e.  The experts follow one
// another and each expert's tiles are spread over all XCDs: their work goes by its rows, and
// whole experts on one XCD left the others waiting (16384 rows of 32 experts, bf16, 4096 x
// 2048: 483 us, against 418).
__device__ __forceinline__ void wgrad_tile(int wg, int per, int tiles_m, int tiles_n, int& e,
                                           int& tm, int& tn) {
  e = wg / per;
  band_order(xcd_order(wg - e * per, per), tiles_m, tiles_n, tm, tn);
}

// Which tile workgroup `wg` of `nwg` computes.  The launch has a workgroup for the largest
// number of tiles that any offsets can give; the count that these give is found here, by
// every wave for itself, 64 groups at a time, and the workgroups past it return false.
// Group 0 is the rows before offsets[0], group E + 1 the ones from offsets[E] on.
// HALF > 0: half a tile (HALF rows or fewer) costs less than a whole one (256 rows 0.72, 64 rows
// of FP32 0.55), and they come last, to fill the last round: a group's last tile where it has no
// more rows; and both halves of each tile of the last round, where these and the others fit into
// one round (bf16, 2304 x 8192 x 4096, 288 tiles: 157 us, 169 with whole tiles).
template <int BM, int HALF>
__device__ inline bool find_tile(const LpArgs& p, int wg, int nwg, TileAt& t) {
  int tm;
  const bool one = p.offsets == nullptr;
  if (HALF == 0 && one) {
    const int tiles_m = (p.rows + BM - 1) / BM, n = tiles_m * p.tiles_n;
    if (wg >= n) return false;
    band_order(xcd_order(wg, n), tiles_m, p.tiles_n, tm, t.tn);
    t.e = 0;
    t.row0 = tm * BM;
    t.row_end = p.rows;
    t.half = false;
    return true;
  }
  const int lane = threadIdx.x & 63;
  const int groups = one ? 1 : p.E + 2;
  int lo = 0, hi = 0, whole = 0, part = 0;  // this lane's group, running counts up to it
  auto load = [&](int base) {
    const int g = base + lane;
    lo = hi = 0;
    if (g < groups) {
      lo = g == 0 ? 0 : clamped_offset(p.offsets, g - 1, p.rows);
      hi = g == groups - 1 ? p.rows : clamped_offset(p.offsets, g, p.rows);
    }
    const int len = max(hi - lo, 0), rest = len % BM;
    part = rest > 0 && rest <= HALF ? 1 : 0;
    whole = len / BM + (rest > 0 ? 1 : 0) - part;
    if (one) return;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int w = __shfl_up(whole, d), q = __shfl_up(part, d);
      if (lane >= d) whole += w, part += q;
    }
  };
  int wholes = 0, parts = 0;
  for (int base = 0; base < groups; base += 64) {
    load(base);
    wholes += __shfl(whole, one ? 0 : 63);
    parts += __shfl(part, one ? 0 : 63);
  }
  int nw = (int)min((int64_t)wholes * p.tiles_n, (int64_t)nwg);
  const int np = (int)min((int64_t)parts * p.tiles_n, (int64_t)(nwg - nw));
  int cut = HALF > 0 ? nw % kCus : 0;  // tiles that are halved
  if (2 * cut + np > kCus) cut = 0;
  nw -= cut;
  if (wg >= nw + np + 2 * cut) return false;
  const bool small = wg >= nw && wg < nw + np, halved = wg >= nw + np;
  t.half = small || halved;
  int id = small ? xcd_order(wg - nw, np)
                 : halved ? nw + (wg - nw - np) / 2 : xcd_order(wg, nw);
  for (int base = 0; base < groups; base += 64) {
    if (groups > 64) load(base);
    const int upto = small ? part : whole;
    const uint64_t past = __ballot((int64_t)upto * p.tiles_n > id);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int before = l ? __shfl(upto, l - 1) : 0;
      const int first = __shfl(lo, l);
      const int g = base + l;
      t.e = one ? 0 : g == 0 || g == p.E + 1 ? -1 : g - 1;
      t.row_end = __shfl(hi, l);
      id -= before * p.tiles_n;
      if (small) {
        t.tn = id;
        t.row0 = first + (t.row_end - first) / BM * BM;
      } else {
        band_order(id, __shfl(upto, l) - before, p.tiles_n, tm, t.tn);
        t.row0 = first + tm * BM;
        if (halved) {
          if ((wg - nw - np) & 1) t.row0 += HALF;
          else t.row_end = min(t.row_end, t.row0 + HALF);
        }
      }
      return true;
    }
    id -= __shfl(upto, 63) * p.tiles_n;
  }
  return false;
}

// Store neighbouring values of one row, of which `n` are inside it, in one store of any
// alignment where all are.  One rounding to the nearest, ties to even.
// OUT: the type, or -1 where it is only known as `any`.
template <int COUNT, int OUT>
__device__ __forceinline__ void store_row(void* C, int64_t at, int n, int any, const float* v) {
  const int type = OUT >= 0 ? OUT : any;
  if (type == GEMM_LP_F32) {
    typedef float group __attribute__((ext_vector_type(4), aligned(4)));
    float* p = (float*)C + at;
    if (n >= COUNT) {
#pragma unroll
      for (int i = 0; i < COUNT; i += 4) *(group*)(p + i) = group{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < COUNT; ++i)
        if (i < n) p[i] = v[i];
    }
    return;
  }
  typedef uint32_t group __attribute__((ext_vector_type(COUNT / 2), aligned(2)));
  group h;
#pragma unroll
  for (int i = 0; i < COUNT; i += 2) {
    uint16_t lo, hi;
    if (type == GEMM_LP_BF16) {
      lo = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
      hi = __builtin_bit_cast(uint16_t, (__bf16)v[i + 1]);
    } else {
      lo = __builtin_bit_cast(uint16_t, (_Float16)v[i]);
      hi = __builtin_bit_cast(uint16_t, (_Float16)v[i + 1]);
    }
    h[i / 2] = (uint32_t)lo | (uint32_t)hi << 16;
  }
  uint16_t* p = (uint16_t*)C + at;
  if (n >= COUNT) {
    *(group*)p = h;
  } else {
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      if (i < n) p[i] = (uint16_t)(h[i / 2] >> (16 * (i & 1)));
  }
}

// Host: a kernel and how it is launched.
using LpKernel = void (*)(LpArgs);

}  // namespace gemmlp

namespace gemmf32 {
void set_last_hip_error(int code);  // what gemm_f32_last_hip_error reports (gemm_f32.hip)
}
