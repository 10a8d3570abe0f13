// Host side of the adapters: argument checks, splits, launches, and their part of the C ABI of
// include/gemm_experts.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ex_adapters.h"
#include "gemm_experts.h"
#include "lp_host.h"

namespace gemmlp {

// Tiles of bm places: the most that any offsets give.
static int64_t place_tiles(int64_t rows, int64_t E, int bm) {
  return rows / bm + std::min<int64_t>(E + 2, rows);
}

// Waves of a workgroup of `down` with places of their own (the others share K): more than one only
// where that leaves a workgroup for every CU, and the adapters have several tiles on average.
static int down_waves(int64_t rows, int64_t E) {
  for (int w = 4; w > 1; w /= 2)
    if (rows >= 16 * w * kCus && rows >= 64 * w * E) return w;
  return 1;
}
// Splits of K: enough workgroups for two a CU where there is not one for each, but 256 columns a
// split.
static int adapter_splits(int64_t rows, int64_t K, int64_t E) {
  const int64_t tiles = std::max<int64_t>(place_tiles(rows, E, 16 * down_waves(rows, E)), 1);
  if (tiles >= kCus) return 1;
  return (int)std::max<int64_t>(
      std::min<int64_t>({(2 * kCus + tiles - 1) / tiles, K / 256, 8}), 1);
}
// Places of a workgroup of `up`.
static int up_places(int64_t rows, int64_t E, int splits) {
  return rows >= 32 * E && splits == 1 ? 64 : 16;
}

// Fragments of the rank of a workgroup of `grad`.
static int grad_fragments(int64_t rank, int bytes) {
  return rank <= 16 ? 1 : rank <= 32 || bytes == 4 ? 2 : 4;
}
static int64_t grad_blocks(int64_t N, int64_t rank, int64_t E, int bytes) {
  const int64_t per = 16 * grad_fragments(rank, bytes);
  return (N + kWaveCols - 1) / kWaveCols * ((rank + per - 1) / per) * E;
}
// Splits of a group's rows in `grad`: enough workgroups for one a CU where the groups are as long
// as the average, but 256 rows a split.
static int grad_splits(int64_t rows, int64_t N, int64_t rank, int64_t E, int bytes) {
  const int64_t wgs = std::max<int64_t>(grad_blocks(N, rank, E, bytes), 1);
  const int64_t each = rows / std::max<int64_t>(E, 1);
  return (int)std::max<int64_t>(
      std::min<int64_t>({(kCus + wgs - 1) / wgs, each / 256, 16}), 1);
}

template <class T, int RW>
static const void* down_kernel(int64_t rank) {
  return rank <= 16   ? (const void*)&ex_adapters_down_kernel<T, 1, RW>
         : rank <= 32 ? (const void*)&ex_adapters_down_kernel<T, 2, RW>
         : rank <= 64 ? (const void*)&ex_adapters_down_kernel<T, 4, RW>
                      : (const void*)&ex_adapters_down_kernel<T, 8, RW>;
}
template <class T>
static const void* down_kernel(int64_t rank, int waves) {
  return waves == 4   ? down_kernel<T, 4>(rank)
         : waves == 2 ? down_kernel<T, 2>(rank)
                      : down_kernel<T, 1>(rank);
}
template <class T, int BM>
static const void* up_kernel(int64_t rank) {
  return rank <= 32   ? (const void*)&ex_adapters_up_kernel<T, 1, BM>
         : rank <= 64 ? (const void*)&ex_adapters_up_kernel<T, 2, BM>
                      : (const void*)&ex_adapters_up_kernel<T, 4, BM>;
}
template <class T>
static const void* up_kernel(int64_t rank, int places) {
  return places == 64 ? up_kernel<T, 64>(rank) : up_kernel<T, 16>(rank);
}
template <class T>
static const void* grad_kernel(int fragments) {
  if constexpr (T::BYTES == 2) {
    if (fragments == 4) return (const void*)&ex_adapters_grad_kernel<T, 4>;
  }
  return fragments == 1 ? (const void*)&ex_adapters_grad_kernel<T, 1>
                        : (const void*)&ex_adapters_grad_kernel<T, 2>;
}
#define BY_TYPE(type, f)                                     \
  ((type) == GEMM_LP_BF16  ? (const void*)f(Bf16)            \
   : (type) == GEMM_LP_F16 ? (const void*)f(F16)             \
                           : (const void*)f(F32))

static bool bad_dims(int64_t rows, int64_t wide, int64_t rank, int64_t E) {
  return rows < 0 || wide < 0 || rank < 0 || E < 0;
}
static bool too_large(int64_t rows, int64_t wide, int64_t E) {
  return rows > kMaxDim || wide > kMaxDim || E > kMaxDim;
}
// (tiles of any launch as a grid of 32-bit threads)
static bool fits_grid(int64_t wgs, int threads) {
  return wgs <= kMaxDim && wgs * threads <= 0xFFFFFFFFLL;
}

static int run_down(int64_t rows, int64_t K, int64_t rank, int64_t E, const int64_t* order,
                    const int32_t* offsets, const void* X, int64_t ldx, const void* A, int64_t lda,
                    int64_t stride_a, const float* scale, float* U, int splits, int type,
                    void* stream) {
  if (bad_dims(rows, K, rank, E)) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (rank > GEMM_ADAPTERS_MAX_RANK || splits < 1 || splits > GEMM_ADAPTERS_MAX_SPLITS) return GEMMF32_ERR_BAD_CONFIG;
  if (ldx < at_least_1(K) || lda < at_least_1(K) || stride_a < 0) return GEMMF32_ERR_BAD_LD;
  if (too_large(rows, K, E)) return GEMMF32_ERR_TOO_LARGE;
  if (rows == 0 || rank == 0 || E == 0) return GEMMF32_OK;
  if (order == nullptr || offsets == nullptr || U == nullptr ||
      (K && (X == nullptr || A == nullptr)))
    return GEMMF32_ERR_NULL_PTR;
  const int b = type_bytes(type);
  if (misaligned(order, 8) || misaligned(offsets, 4) || misaligned(scale, 4) || misaligned(U, 16) ||
      misaligned(X, b) || misaligned(A, b))
    return GEMMF32_ERR_MISALIGNED;
  const int64_t ldu = u_columns((int)rank);
  Range u, in[5];
  if (!byte_range(U, splits, rows * ldu, rows, ldu, ldu, 4, &u) ||
      !byte_range(order, 1, 0, 1, rows, rows, 8, &in[0]) ||
      !byte_range(offsets, 1, 0, 1, E + 1, E + 1, 4, &in[1]) ||
      (scale && !byte_range(scale, 1, 0, 1, E, E, 4, &in[2])) ||
      (K && (!byte_range(X, 1, 0, rows, K, ldx, b, &in[3]) ||
             !byte_range(A, E, stride_a, rank, K, lda, b, &in[4]))))
    return GEMMF32_ERR_TOO_LARGE;
  for (const Range& r : in)
    if (overlap(u, r)) return GEMMF32_ERR_ALIAS;
  AdapterArgs a{};
  a.X = X, a.W = A, a.offsets = offsets, a.order = order, a.scale = scale, a.U = U;
  a.ldx = ldx, a.ldw = lda, a.stride_w = stride_a;
  a.rows = (int)rows, a.K = (int)K, a.E = (int)E, a.rank = (int)rank, a.ldu = (int)ldu;
  a.splits = splits;
  // (a multiple of the steps that four waves take at once)
  const int64_t unit = 4 * 128 / b;
  a.k_chunk = (int)((K + splits * unit - 1) / (splits * unit) * unit);
  const int waves = down_waves(rows, E);
  const int64_t wgs = place_tiles(rows, E, 16 * waves) * splits;
  if (!fits_grid(wgs, kDownThreads)) return GEMMF32_ERR_TOO_LARGE;
#define DOWN(T) down_kernel<T>(rank, waves)
  return launch(BY_TYPE(type, DOWN), dim3((unsigned)wgs), kDownThreads, &a, stream);
#undef DOWN
}

static int run_up(int64_t rows, int64_t N, int64_t rank, int64_t E, const int64_t* order,
                  const int32_t* offsets, const float* U, int splits, const void* B, int64_t ldb,
                  int64_t stride_b, const void* Y, int64_t ldy, void* OUT, int64_t ldo, int type,
                  void* stream) {
  if (bad_dims(rows, N, rank, E)) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (rank > GEMM_ADAPTERS_MAX_RANK || splits < 1 || splits > GEMM_ADAPTERS_MAX_SPLITS) return GEMMF32_ERR_BAD_CONFIG;
  if (ldb < at_least_1(N) || stride_b < 0 || (Y && ldy < at_least_1(N)) || ldo < at_least_1(N))
    return GEMMF32_ERR_BAD_LD;
  if (too_large(rows, N, E)) return GEMMF32_ERR_TOO_LARGE;
  if (rows == 0 || N == 0) return GEMMF32_OK;
  const bool reads = rank > 0 && E > 0;
  if (order == nullptr || offsets == nullptr || OUT == nullptr ||
      (reads && (U == nullptr || B == nullptr)))
    return GEMMF32_ERR_NULL_PTR;
  const int b = type_bytes(type);
  if (misaligned(order, 8) || misaligned(offsets, 4) || misaligned(U, 16) || misaligned(B, b) ||
      misaligned(Y, b) || misaligned(OUT, b))
    return GEMMF32_ERR_MISALIGNED;
  const int64_t ldu = u_columns((int)rank);
  Range o, in[5];
  if (!byte_range(OUT, 1, 0, rows, N, ldo, b, &o) ||
      !byte_range(order, 1, 0, 1, rows, rows, 8, &in[0]) ||
      !byte_range(offsets, 1, 0, 1, E + 1, E + 1, 4, &in[1]) ||
      (reads && (!byte_range(U, splits, rows * ldu, rows, ldu, ldu, 4, &in[2]) ||
                 !byte_range(B, E, stride_b, rank, N, ldb, b, &in[3]))) ||
      (Y && !byte_range(Y, 1, 0, rows, N, ldy, b, &in[4])))
    return GEMMF32_ERR_TOO_LARGE;
  for (const Range& r : in)
    if (overlap(o, r)) return GEMMF32_ERR_ALIAS;
  AdapterArgs a{};
  a.W = B, a.C = OUT, a.offsets = offsets, a.order = order, a.U = (float*)U, a.Y = Y;
  a.ldw = ldb, a.stride_w = stride_b, a.ldc = ldo, a.ldy = ldy;
  a.rows = (int)rows, a.N = (int)N, a.E = (int)E, a.rank = (int)rank, a.ldu = (int)ldu;
  a.splits = splits, a.tiles_n = (int)((N + kUpCols - 1) / kUpCols);
  // (rank 0: no place has an adapter)
  if (!reads) a.E = 0;
  const int places = up_places(rows, E, splits);
  int64_t wgs;
  if (__builtin_mul_overflow(place_tiles(rows, E, places), (int64_t)a.tiles_n, &wgs) ||
      !fits_grid(wgs, kUpThreads))
    return GEMMF32_ERR_TOO_LARGE;
#define UP(T) up_kernel<T>(rank, places)
  return launch(BY_TYPE(type, UP), dim3((unsigned)wgs), kUpThreads, &a, stream);
#undef UP
}

static int64_t grad_workspace(int64_t rows, int64_t N, int64_t rank, int64_t E, int bytes) {
  const int s = grad_splits(rows, N, rank, E, bytes);
  return s > 1 ? (int64_t)s * E * rank * N * 4 : 0;
}

static int run_adapters_grad(int64_t rows, int64_t N, int64_t rank, int64_t E,
                             const int64_t* order, const int32_t* offsets, const float* U,
                             int splits, const void* X, int64_t ldx, void* D, int64_t ldd,
                             int64_t stride_d, void* workspace, int64_t workspace_bytes, int type,
                             void* stream) {
  if (bad_dims(rows, N, rank, E)) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (rank > GEMM_ADAPTERS_MAX_RANK || splits < 1 || splits > GEMM_ADAPTERS_MAX_SPLITS) return GEMMF32_ERR_BAD_CONFIG;
  if (ldx < at_least_1(N) || ldd < at_least_1(N)) return GEMMF32_ERR_BAD_LD;
  if (too_large(rows, N, E)) return GEMMF32_ERR_TOO_LARGE;
  if (N == 0 || rank == 0 || E == 0) return GEMMF32_OK;
  const int b = type_bytes(type);
  const bool reads = rows > 0;
  const int64_t ldu = u_columns((int)rank);
  Range out[2], one, in[4];
  if (D == nullptr || offsets == nullptr ||
      (reads && (order == nullptr || U == nullptr || X == nullptr)))
    return GEMMF32_ERR_NULL_PTR;
  if (misaligned(D, b) || misaligned(X, b) || misaligned(U, 16) || misaligned(order, 8) ||
      misaligned(offsets, 4) || misaligned(workspace, 8))
    return GEMMF32_ERR_MISALIGNED;
  if (!byte_range(D, E, stride_d, rank, N, ldd, b, &out[0]) ||
      !byte_range(D, 1, 0, rank, N, ldd, b, &one) ||
      !byte_range(offsets, 1, 0, 1, E + 1, E + 1, 4, &in[0]) ||
      (reads && (!byte_range(order, 1, 0, 1, rows, rows, 8, &in[1]) ||
                 !byte_range(U, splits, rows * ldu, rows, ldu, ldu, 4, &in[2]) ||
                 !byte_range(X, 1, 0, rows, N, ldx, b, &in[3]))))
    return GEMMF32_ERR_TOO_LARGE;
  // each expert's D has to end where the next begins, or it would be written twice
  if (E > 1 && (stride_d < 0 || (uint64_t)stride_d * b < (uint64_t)(one.hi - one.lo)))
    return GEMMF32_ERR_BAD_LD;
  const int64_t need = grad_workspace(rows, N, rank, E, b);  // (fits: D's extent does)
  if (workspace_bytes < need) return GEMMF32_ERR_BAD_LD;
  if (need && workspace == nullptr) return GEMMF32_ERR_NULL_PTR;
  if (need && !byte_range(workspace, 1, 0, 1, need, need, 1, &out[1])) return GEMMF32_ERR_TOO_LARGE;
  if (overlap(out[0], out[1])) return GEMMF32_ERR_ALIAS;
  for (const Range& r : in)
    if (overlap(out[0], r) || overlap(out[1], r)) return GEMMF32_ERR_ALIAS;
  AdapterArgs a{};
  a.X = X, a.C = D, a.offsets = offsets, a.order = order, a.U = (float*)U;
  a.part = (float*)workspace, a.ldx = ldx, a.ldc = ldd, a.stride_c = stride_d;
  a.rows = (int)rows, a.N = (int)N, a.E = (int)E, a.rank = (int)rank, a.ldu = (int)ldu;
  a.splits = splits, a.tiles_n = (int)((N + kWaveCols - 1) / kWaveCols);
  a.row_splits = grad_splits(rows, N, rank, E, b);
  const int fragments = grad_fragments(rank, b);
  const int threads = 64 * (fragments <= 2 ? GradShape<1>::WAVES : GradShape<4>::WAVES);
  int64_t wgs;
  if (__builtin_mul_overflow(grad_blocks(N, rank, E, b), (int64_t)a.row_splits, &wgs) ||
      !fits_grid(wgs, threads))
    return GEMMF32_ERR_TOO_LARGE;
#define GRAD(T) grad_kernel<T>(fragments)
  if (const int rc = launch(BY_TYPE(type, GRAD), dim3((unsigned)wgs), threads, &a, stream)) return rc;
#undef GRAD
  if (a.row_splits == 1) return GEMMF32_OK;
  const int64_t sums = (E * rank * ((N + 7) / 8) + 255) / 256;
  if (!fits_grid(sums, 256)) return GEMMF32_ERR_TOO_LARGE;
#define SUM(T) &ex_adapters_sum_kernel<T>
  return launch(BY_TYPE(type, SUM), dim3((unsigned)sums), 256, &a, stream);
#undef SUM
}

}  // namespace gemmlp

extern "C" {

int gemm_adapters_down(int64_t rows, int64_t K, int64_t rank, int64_t E, const int64_t* order,
                       const int32_t* offsets, const void* X, int64_t ldx, const void* A,
                       int64_t lda, int64_t stride_a, const float* scale, float* U, int splits,
                       int type, void* stream) {
  return gemmlp::run_down(rows, K, rank, E, order, offsets, X, ldx, A, lda, stride_a, scale, U,
                          splits, type, stream);
}

int gemm_adapters_up(int64_t rows, int64_t N, int64_t rank, int64_t E, const int64_t* order,
                     const int32_t* offsets, const float* U, int splits, const void* B,
                     int64_t ldb, int64_t stride_b, const void* Y, int64_t ldy, void* OUT,
                     int64_t ldo, int type, void* stream) {
  return gemmlp::run_up(rows, N, rank, E, order, offsets, U, splits, B, ldb, stride_b, Y, ldy, OUT,
                        ldo, type, stream);
}

int gemm_adapters_grad(int64_t rows, int64_t N, int64_t rank, int64_t E, const int64_t* order,
                       const int32_t* offsets, const float* U, int splits, const void* X,
                       int64_t ldx, void* D, int64_t ldd, int64_t stride_d, void* workspace,
                       int64_t workspace_bytes, int type, void* stream) {
  return gemmlp::run_adapters_grad(rows, N, rank, E, order, offsets, U, splits, X, ldx, D, ldd,
                                   stride_d, workspace, workspace_bytes, type, stream);
}

int gemm_adapters_splits(int64_t rows, int64_t K, int64_t rank, int64_t E) {
  if (gemmlp::bad_dims(rows, K, rank, E)) return GEMMF32_ERR_NEGATIVE_DIM;
  if (rank > GEMM_ADAPTERS_MAX_RANK) return GEMMF32_ERR_BAD_CONFIG;
  if (gemmlp::too_large(rows, K, E)) return GEMMF32_ERR_TOO_LARGE;
  return gemmlp::adapter_splits(rows, K, E);
}

int64_t gemm_adapters_grad_workspace(int64_t rows, int64_t N, int64_t rank, int64_t E, int type) {
  if (gemmlp::bad_dims(rows, N, rank, E)) return GEMMF32_ERR_NEGATIVE_DIM;
  if (rank > GEMM_ADAPTERS_MAX_RANK) return GEMMF32_ERR_BAD_CONFIG;
  if (gemmlp::too_large(rows, N, E)) return GEMMF32_ERR_TOO_LARGE;
  if (!gemmlp::known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  return gemmlp::grad_workspace(rows, N, rank, E, gemmlp::type_bytes(type));
}

}  // extern "C"
