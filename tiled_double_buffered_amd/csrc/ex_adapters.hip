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

// Whether `down` takes 64 places a workgroup or 16: the adapter's lines are read for every tile, so that
// few places pay where these are few: few columns, or a low rank, whose rows' own bytes decide.  From
// 10000 rows on (5000 past rank 64) tiles of 64 fill the chip without splits of K and their join.
// (Over 3104 sizes, 32 to 20000 rows, 256 to 11008 columns, ranks 16 to 128, 1 to 64 adapters, bf16 and FP32,
// the choice is 1.8 % slower than the better one in the mean and 6 % or more for a tenth of them; always
// 16 17 %, always 64 14 %.  bf16, with 16 and 64, in us with the join: 8192 x 4096, rank 32, four uneven adapters, 28 and 22; rank
// 16 22 and 21; 4096 x 4096, rank 16, 14 and 17, rank 64 26 and 20; 8192 x 1024, rank 64, 12 and 14; 16384
// x 1024 22 and 17; 1024 x 11008, rank 128, 34 and 21.)
static bool down_wide(int64_t rows, int64_t K, int64_t rank) {
  if (rows >= (rank > 64 ? 5000 : 10000)) return true;
  const int64_t fragments = rank <= 32 ? 32 : rank <= 64 ? 64 : 128;
  return rows >= (rank > 16 ? 1024 : 5000) && fragments * K > 65536;
}
static int64_t down_tiles(int64_t rows, int64_t K, int64_t rank, int64_t E) {
  return place_tiles(rows, E, down_wide(rows, K, rank) ? kWidePlaces : 16);
}
// Splits of K: enough workgroups for two a CU where there are none for each, but 256 columns a split.
static int adapter_splits(int64_t rows, int64_t K, int64_t rank, int64_t E) {
  const int64_t tiles = std::max<int64_t>(down_tiles(rows, K, rank, E), 1);
  if (tiles >= kCus * 3 / 4) return 1;
  return (int)std::max<int64_t>(std::min<int64_t>({2 * kCus / tiles, K / 256, 8}), 1);
}
// Places of a workgroup of `up`, a wave, up to rank 32: those that take the least time, as the rounds
// of waves (four of a SIMD) and a round's places, of which its start is worth about 24.  (504 sizes, 128
// to 16384 rows, 1024 to 11008 columns, 1 to 64 adapters: 1.2 % slower than the best in the mean, FP32 1.8;
// 14 % at most, where a tile more makes one more round by this count and not in fact.  Always 16: 2.4 to
// 2.9 %, 32 8 to 12.  bf16, rank 16, four uneven adapters, in us with 16, 32 and 64: 1024 x 4096 7.4, 8.0
// and 10; 4096 x 4096 20, 20 and 21; 8192 x 4096 37, 35 and 37; 4096 x 11008 47, 45 and 47.  A count of its
// own for fp16 and FP32, whose registers leave three and two waves, gains 0.2 and 0.6 % in the mean.)
static int up_places(int64_t rows, int64_t N, int64_t E) {
  int best = 16;
  int64_t least = 0;
  for (int bm = 16; bm <= 64; bm *= 2) {
    const int64_t tiles = (rows + bm - 1) / bm + std::min(E, rows) / 2;
    const int64_t rounds = (tiles * ((N + kWaveCols - 1) / kWaveCols) + 16 * kCus - 1) / (16 * kCus);
    if (bm == 16 || rounds * (bm + 24) < least) best = bm, least = rounds * (bm + 24);
  }
  return best;
}

// Fragments of the rank of a workgroup of `grad`.
static int grad_fragments(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : 4; }
static int64_t grad_blocks(int64_t N, int64_t rank) {
  const int64_t per = 16 * grad_fragments(rank), columns = grad_columns((int)rank);
  return (N + columns - 1) / columns * ((rank + per - 1) / per);
}
// Waves of a workgroup of `grad`: four past rank 32, of which two workgroups fit on a CU, and where the adapters have
// fewer places than eight take in a turn.
static int grad_waves(int64_t rows, int64_t rank, int64_t E) {
  return rank > 32 || rows < 256 * E ? 4 : 8;
}
// Places of a run in `grad` for gradients of so many workgroups a run together: so many that there are
// two workgroups for each CU and four runs (one where a run has as many), but a turn of the waves at
// least.  (Four, as with fewer the longest adapter decides: 16384 x 4096 of eight uneven ones, rank 128,
// 231 us, 255 without, when it was chosen.)
static int64_t grad_run(int64_t rows, int64_t blocks, int waves) {
  const int64_t per =
      blocks > 2 * kCus ? 1 : std::max<int64_t>(2 * kCus / std::max<int64_t>(blocks, 1), 4);
  const int64_t turn = 32 * waves;
  return std::max<int64_t>(((rows + per - 1) / per + turn - 1) / turn * turn, turn);
}
// The most runs that there can be.
static int64_t grad_runs(int64_t rows, int64_t E, int64_t run) { return rows / run + E; }
// Runs of the adapters that have several, the most that there can be: an adapter of more than `run`
// places has fewer than twice as many runs as its places fill.
static int64_t grad_slots(int64_t rows, int64_t E, int64_t run) {
  return std::min(grad_runs(rows, E, run), 2 * rows / run);
}

template <class T>
static const void* down_kernel(int64_t rank, bool wide) {
  if (wide)
    return rank <= 16   ? (const void*)&ex_adapters_down_wide_kernel<T, 1>
           : rank <= 32 ? (const void*)&ex_adapters_down_wide_kernel<T, 2>
           : rank <= 64 ? (const void*)&ex_adapters_down_wide_kernel<T, 4>
                        : (const void*)&ex_adapters_down_wide_kernel<T, 8>;
  return rank <= 16   ? (const void*)&ex_adapters_down_kernel<T, 1>
         : rank <= 32 ? (const void*)&ex_adapters_down_kernel<T, 2>
         : rank <= 64 ? (const void*)&ex_adapters_down_kernel<T, 4>
                      : (const void*)&ex_adapters_down_kernel<T, 8>;
}
template <class T>
static const void* up_kernel(int64_t rank, int places) {
  return rank > 32       ? (const void*)&ex_adapters_up_deep_kernel<T>
         : places == 64 ? (const void*)&ex_adapters_up_kernel<T, 64>
         : places == 32 ? (const void*)&ex_adapters_up_kernel<T, 32>
                        : (const void*)&ex_adapters_up_kernel<T, 16>;
}
template <class T>
static const void* grad_kernel(int fragments, int waves) {
  if (fragments == 4) return (const void*)&ex_adapters_grad_kernel<T, 4, 4>;
  if (waves == 4)
    return fragments == 1 ? (const void*)&ex_adapters_grad_kernel<T, 1, 4>
                          : (const void*)&ex_adapters_grad_kernel<T, 2, 4>;
  return fragments == 1 ? (const void*)&ex_adapters_grad_kernel<T, 1, 8>
                        : (const void*)&ex_adapters_grad_kernel<T, 2, 8>;
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
                    int64_t stride_a, const float* scale, float* U, int splits, int join,
                    int type, void* stream) {
  if (bad_dims(rows, K, rank, E)) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (rank > GEMM_ADAPTERS_MAX_RANK || splits < 1 || splits > GEMM_ADAPTERS_MAX_SPLITS)
    return GEMMF32_ERR_BAD_CONFIG;
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
  const bool wide = down_wide(rows, K, rank);
  const int threads = wide ? kWideThreads : kDownThreads;
  const int64_t wgs = down_tiles(rows, K, rank, E) * splits;
  if (K < kLeastWide) {
    const int64_t few = place_tiles(rows, E, 16) * splits;
    if (!fits_grid(few, 256)) return GEMMF32_ERR_TOO_LARGE;
#define FEW(T) &ex_adapters_down_few_kernel<T>
    return launch(BY_TYPE(type, FEW), dim3((unsigned)few), 256, &a, stream);
#undef FEW
  }
  if (!fits_grid(wgs, threads)) return GEMMF32_ERR_TOO_LARGE;
#define DOWN(T) down_kernel<T>(rank, wide)
  if (const int rc = launch(BY_TYPE(type, DOWN), dim3((unsigned)wgs), threads, &a, stream)) return rc;
#undef DOWN
  if (!join || splits == 1) return GEMMF32_OK;
  const int64_t sums = (rows * ldu / 4 + 255) / 256;
  if (!fits_grid(sums, 256)) return GEMMF32_ERR_TOO_LARGE;
  return launch((const void*)&ex_adapters_join_kernel, dim3((unsigned)sums), 256, &a, stream);
}

static int run_up(int64_t rows, int64_t N, int64_t rank, int64_t E, const int64_t* order,
                  const int32_t* offsets, const float* U, int splits, const void* B, int64_t ldb,
                  int64_t stride_b, const void* Y, int64_t ldy, void* OUT, int64_t ldo, int type,
                  void* stream) {
  if (bad_dims(rows, N, rank, E)) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (rank > GEMM_ADAPTERS_MAX_RANK || splits < 1 || splits > GEMM_ADAPTERS_MAX_SPLITS)
    return GEMMF32_ERR_BAD_CONFIG;
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
  a.splits = splits, a.tiles_n = (int)((N + kWaveCols - 1) / kWaveCols);
  // (rank 0: no place has an adapter)
  if (!reads) a.E = 0;
  if (N < kLeastWide) {
    const int64_t few = place_tiles(rows, a.E, 16);
    if (!fits_grid(few, 256)) return GEMMF32_ERR_TOO_LARGE;
#define FEW(T) &ex_adapters_up_few_kernel<T>
    return launch(BY_TYPE(type, FEW), dim3((unsigned)few), 256, &a, stream);
#undef FEW
  }
  const int places = rank > 32 ? 64 : up_places(rows, N, E), threads = rank > 32 ? 256 : 64;
  int64_t wgs;
  if (__builtin_mul_overflow(place_tiles(rows, E, places), (int64_t)a.tiles_n, &wgs) ||
      !fits_grid(wgs, threads))
    return GEMMF32_ERR_TOO_LARGE;
#define UP(T) up_kernel<T>(rank, places)
  return launch(BY_TYPE(type, UP), dim3((unsigned)wgs), threads, &a, stream);
#undef UP
}

// One of the gradients of a step, N columns wide.
struct GradSide {
  int64_t N;
  const float* U;
  int splits;
  const void* X;
  int64_t ldx;
  void* D;
  int64_t ldd, stride_d;
  bool wide() const { return N >= kLeastWide; }
};
static int64_t side_blocks(int64_t N, int64_t rank) {
  return N >= kLeastWide ? grad_blocks(N, rank) : 0;
}
// Bytes of a gradient's slots: of the runs whose sums another launch adds.  (Several runs there are
// only of 65536 columns or fewer, so that 64 bits hold them.)
static int64_t side_workspace(int64_t rows, int64_t N, int64_t rank, int64_t E, int64_t run) {
  return rows > run && N >= kLeastWide ? grad_slots(rows, E, run) * rank * N * 4 : 0;
}

static int run_adapters_grad(int64_t rows, int64_t rank, int64_t E, const int64_t* order,
                             const int32_t* offsets, const GradSide (&sides)[2], void* workspace,
                             int64_t workspace_bytes, int type, void* stream) {
  for (const GradSide& s : sides)
    if (bad_dims(rows, s.N, rank, E)) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (rank > GEMM_ADAPTERS_MAX_RANK) return GEMMF32_ERR_BAD_CONFIG;
  if (rank == 0 || E == 0) return GEMMF32_OK;
  const int b = type_bytes(type);
  const bool reads = rows > 0;
  const int64_t ldu = u_columns((int)rank);
  const int waves = grad_waves(rows, rank, E), threads = 64 * waves;
  const int64_t run =
      grad_run(rows, side_blocks(sides[0].N, rank) + side_blocks(sides[1].N, rank), waves);
  Range out[3], in[6];
  int64_t need = 0;
  for (int i = 0; i < 2; ++i) {
    const GradSide& s = sides[i];
    if (s.N == 0) continue;
    if (s.splits < 1 || s.splits > GEMM_ADAPTERS_MAX_SPLITS) return GEMMF32_ERR_BAD_CONFIG;
    if (s.ldx < s.N || s.ldd < s.N) return GEMMF32_ERR_BAD_LD;
    if (too_large(rows, s.N, E)) return GEMMF32_ERR_TOO_LARGE;
    if (s.D == nullptr || offsets == nullptr ||
        (reads && (order == nullptr || s.U == nullptr || s.X == nullptr)))
      return GEMMF32_ERR_NULL_PTR;
    if (misaligned(s.D, b) || misaligned(s.X, b) || misaligned(s.U, 16))
      return GEMMF32_ERR_MISALIGNED;
    Range one;
    if (!byte_range(s.D, E, s.stride_d, rank, s.N, s.ldd, b, &out[i]) ||
        !byte_range(s.D, 1, 0, rank, s.N, s.ldd, b, &one) ||
        (reads && (!byte_range(s.U, s.splits, rows * ldu, rows, ldu, ldu, 4, &in[2 * i]) ||
                   !byte_range(s.X, 1, 0, rows, s.N, s.ldx, b, &in[2 * i + 1]))))
      return GEMMF32_ERR_TOO_LARGE;
    // each expert's D has to end where the next begins, or it would be written twice
    if (E > 1 && (s.stride_d < 0 || (uint64_t)s.stride_d * b < (uint64_t)(one.hi - one.lo)))
      return GEMMF32_ERR_BAD_LD;
    need += side_workspace(rows, s.N, rank, E, run);
  }
  if (sides[0].N == 0 && sides[1].N == 0) return GEMMF32_OK;
  if (misaligned(order, 8) || misaligned(offsets, 4) || misaligned(workspace, 8))
    return GEMMF32_ERR_MISALIGNED;
  if (workspace_bytes < need) return GEMMF32_ERR_BAD_LD;
  if (need && workspace == nullptr) return GEMMF32_ERR_NULL_PTR;
  if ((need && !row_range(workspace, need, 1, &out[2])) || !row_range(offsets, E + 1, 4, &in[4]) ||
      (reads && !row_range(order, rows, 8, &in[5])))
    return GEMMF32_ERR_TOO_LARGE;
  if (any_overlap(out, in)) return GEMMF32_ERR_ALIAS;

  const int fragments = grad_fragments(rank), columns = grad_columns((int)rank);
  GradArgs wide{};
  int64_t wgs[2] = {}, sums[2] = {};
  int count = 0;
  float* part = (float*)workspace;
  for (const GradSide& s : sides) {
    if (s.N == 0) continue;
    AdapterArgs a{};
    a.X = s.X, a.C = s.D, a.offsets = offsets, a.order = order, a.U = (float*)s.U;
    a.part = part, a.ldx = s.ldx, a.ldc = s.ldd, a.stride_c = s.stride_d;
    a.rows = (int)rows, a.N = (int)s.N, a.E = (int)E, a.rank = (int)rank, a.ldu = (int)ldu;
    a.splits = s.splits, a.tiles_n = (int)((s.N + columns - 1) / columns);
    a.run = (int)run, a.slots = (int)grad_slots(rows, E, run);
    if (s.wide()) {
      if (__builtin_mul_overflow(side_blocks(s.N, rank), grad_runs(rows, E, run), &wgs[count]))
        return GEMMF32_ERR_TOO_LARGE;
      sums[count] = E * ((rank * ((s.N + 7) / 8) + 255) / 256);
      part += side_workspace(rows, s.N, rank, E, run) / 4;
      wide.set[count++] = a;
      continue;
    }
    if (!fits_grid(E * rank, 256)) return GEMMF32_ERR_TOO_LARGE;
#define FEW(T) &ex_adapters_grad_few_kernel<T>
    if (const int rc = launch(BY_TYPE(type, FEW), dim3((unsigned)(E * rank)), 256, &a, stream))
      return rc;
#undef FEW
  }
  if (count == 0) return GEMMF32_OK;
  if (wgs[0] > kMaxDim || wgs[1] > kMaxDim || !fits_grid(wgs[0] + wgs[1], threads) ||
      !fits_grid(sums[0] + sums[1], 256))
    return GEMMF32_ERR_TOO_LARGE;
  wide.wgs = (int)wgs[0];
#define GRAD(T) grad_kernel<T>(fragments, waves)
  if (const int rc = launch(BY_TYPE(type, GRAD), dim3((unsigned)(wgs[0] + wgs[1])), threads, &wide,
                            stream))
    return rc;
#undef GRAD
  if (rows <= run) return GEMMF32_OK;  // (one run each)
  wide.wgs = (int)sums[0];
#define SUM(T) &ex_adapters_sum_kernel<T>
  return launch(BY_TYPE(type, SUM), dim3((unsigned)(sums[0] + sums[1])), 256, &wide, stream);
#undef SUM
}

}  // namespace gemmlp

extern "C" {

int gemm_adapters_down(int64_t rows, int64_t K, int64_t rank, int64_t E, const int64_t* order,
                       const int32_t* offsets, const void* X, int64_t ldx, const void* A,
                       int64_t lda, int64_t stride_a, const float* scale, float* U, int splits,
                       int join, int type, void* stream) {
  return gemmlp::run_down(rows, K, rank, E, order, offsets, X, ldx, A, lda, stride_a, scale, U,
                          splits, join, type, stream);
}

int gemm_adapters_up(int64_t rows, int64_t N, int64_t rank, int64_t E, const int64_t* order,
                     const int32_t* offsets, const float* U, int splits, const void* B,
                     int64_t ldb, int64_t stride_b, const void* Y, int64_t ldy, void* OUT,
                     int64_t ldo, int type, void* stream) {
  return gemmlp::run_up(rows, N, rank, E, order, offsets, U, splits, B, ldb, stride_b, Y, ldy, OUT,
                        ldo, type, stream);
}

int gemm_adapters_grad(int64_t rows, int64_t rank, int64_t E, const int64_t* order,
                       const int32_t* offsets, int64_t K, const float* V, int v_splits,
                       const void* X, int64_t ldx, void* DA, int64_t ldda, int64_t stride_da,
                       int64_t N, const float* U, int u_splits, const void* DOUT, int64_t ldd,
                       void* DB, int64_t lddb, int64_t stride_db, void* workspace,
                       int64_t workspace_bytes, int type, void* stream) {
  return gemmlp::run_adapters_grad(rows, rank, E, order, offsets,
                                   {{K, V, v_splits, X, ldx, DA, ldda, stride_da},
                                    {N, U, u_splits, DOUT, ldd, DB, lddb, stride_db}},
                                   workspace, workspace_bytes, type, stream);
}

int gemm_adapters_splits(int64_t rows, int64_t K, int64_t rank, int64_t E) {
  if (gemmlp::bad_dims(rows, K, rank, E)) return GEMMF32_ERR_NEGATIVE_DIM;
  if (rank > GEMM_ADAPTERS_MAX_RANK) return GEMMF32_ERR_BAD_CONFIG;
  if (gemmlp::too_large(rows, K, E)) return GEMMF32_ERR_TOO_LARGE;
  return gemmlp::adapter_splits(rows, K, rank, E);
}

int64_t gemm_adapters_grad_workspace(int64_t rows, int64_t K, int64_t N, int64_t rank, int64_t E,
                                     int type) {
  using namespace gemmlp;
  if (bad_dims(rows, K, rank, E) || N < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (rank > GEMM_ADAPTERS_MAX_RANK) return GEMMF32_ERR_BAD_CONFIG;
  if (too_large(rows, std::max(K, N), E)) return GEMMF32_ERR_TOO_LARGE;
  const int64_t run = grad_run(rows, side_blocks(K, rank) + side_blocks(N, rank),
                               grad_waves(rows, rank, E));
  return side_workspace(rows, K, rank, E, run) + side_workspace(rows, N, rank, E, run);
}

}  // extern "C"
