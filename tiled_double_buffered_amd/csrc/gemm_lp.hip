// Host side of the low-precision and expert-grouped products: argument checks, the choice of
// a kernel, launches, and the C ABI of include/gemm_lp.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "gemm_lp.h"
#include "lp_common.h"
#include "lp_quantize.h"
#include "lp_units.h"

namespace gemmlp {

constexpr int64_t kMaxDim = 2147483647LL - 1024;  // keeps tile-end arithmetic in int32
constexpr int64_t kMaxExtent = (int64_t)1 << 61;   // bytes one operand may span
constexpr int64_t kMaxScaleLd = (int64_t)1 << 22;  // 256 rows of scales in 32-bit offsets

// Byte range [lo, hi) of `count` blocks of rows x cols values of `bytes` bytes, row stride ld
// and block stride `stride` (elements).  False where it passes kMaxExtent or wraps.
struct Range {
  uintptr_t lo = 0, hi = 0;
};
static bool byte_range(const void* p, int64_t count, int64_t stride, int64_t rows, int64_t cols,
                       int64_t ld, int64_t bytes, Range* r) {
  int64_t e, s;
  if (__builtin_mul_overflow(rows - 1, ld, &e) || __builtin_add_overflow(e, cols, &e) ||
      __builtin_mul_overflow(count - 1, stride, &s) || __builtin_add_overflow(e, s, &e) ||
      __builtin_mul_overflow(e, bytes, &e) || e > kMaxExtent)
    return false;
  r->lo = (uintptr_t)p;
  return !__builtin_add_overflow(r->lo, (uintptr_t)e, &r->hi);
}
static bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

static bool known_type(int t) { return t == GEMM_LP_BF16 || t == GEMM_LP_F16 || t == GEMM_LP_F32; }
static bool misaligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) != 0; }
static int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }
static int64_t at_least_1(int64_t n) { return n > 1 ? n : 1; }

static int launch(const void* fn, dim3 grid, int threads, void* args, void* stream) {
  void* list[] = {args};
  const hipError_t err =
      hipLaunchKernel(fn, grid, dim3((unsigned)threads), list, 0, (hipStream_t)stream);
  if (err != hipSuccess) {
    gemmf32::set_last_hip_error((int)err);
    return GEMMF32_ERR_HIP;
  }
  return GEMMF32_OK;
}

// Workgroups of a row product with BM x BN tiles: the most tiles that any offsets give.  A
// group adds at most one partly filled tile to its rows' whole ones, and a group without
// rows none.
static int64_t row_tiles(const LpArgs& a, int64_t BM, int64_t BN) {
  const int64_t m = a.offsets == nullptr
                        ? (a.rows + BM - 1) / BM
                        : a.rows / BM + std::min<int64_t>((int64_t)a.E + 2, a.rows);
  return m * ((a.N + BN - 1) / BN);
}

static LpKernel pipe_kernel(int unit, int tile, bool staged) {
  switch (unit) {
    case 0: return pipe_kernel_0(tile, staged);
    case 1: return pipe_kernel_1(tile, staged);
    case 2: return pipe_kernel_2(tile, staged);
    case 3: return pipe_kernel_3(tile, staged);
    case 4: return pipe_kernel_4(tile, staged);
    case 5: return pipe_kernel_5(tile, staged);
    case 6: return pipe_kernel_6(tile, staged);
    case 7: return pipe_kernel_7(tile, staged);
    case 8: return pipe_kernel_8(tile, staged);
    case 9: return pipe_kernel_9(tile, staged);
    case 10: return pipe_kernel_10(tile, staged);
    default: return pipe_kernel_11(tile, staged);
  }
}

// What half a tile of a row product costs, where it is computed in halves (lp_deep.h, and the
// 64-row tiles of FP32); 1 where it is not.
static double half_cost(int unit, int tile) {
  if (tile == kTile256) return 0.72;
  return tile != kTile128 && (unit == 6 || unit == 7) ? 0.55 : 1.0;
}

static int launch_rows(int unit, int tile, bool staged, LpArgs a, void* stream) {
  const TileSize& s = kTiles[tile];
  // (half a round more where the last round's tiles may be halved)
  const int64_t wgs = row_tiles(a, s.bm, s.bn) + (half_cost(unit, tile) < 1 ? kCus / 2 : 0);
  if (wgs * s.threads > 0xFFFFFFFFLL || wgs > kMaxDim) return GEMMF32_ERR_TOO_LARGE;
  a.tiles_n = (a.N + s.bn - 1) / s.bn;
  return launch((const void*)pipe_kernel(unit, tile, staged), dim3((unsigned)wgs), s.threads, &a,
                stream);
}

static int launch_wgrad(int unit, int tile, bool staged, LpArgs a, void* stream) {
  const TileSize& s = kTiles[tile];
  const int64_t tm = (a.M + s.bm - 1) / s.bm, tn = (a.N + s.bn - 1) / s.bn;
  int64_t wgs;
  if (__builtin_mul_overflow(tm * tn, (int64_t)a.E, &wgs) || wgs > kMaxDim ||
      wgs * s.threads > 0xFFFFFFFFLL)
    return GEMMF32_ERR_TOO_LARGE;
  a.tiles_n = (int)tn;
  return launch((const void*)pipe_kernel(unit, tile, staged), dim3((unsigned)wgs), s.threads, &a,
                stream);
}

// Whether an operand can be copied in words: rows and experts that start at multiples of four
// bytes, and 256 rows (or k rows) within the 32-bit offsets of a copy.
static bool word_rows(const void* p, int64_t ld, int64_t stride, int bytes) {
  return misaligned(p, 4) == false && ld * bytes % 4 == 0 && stride * bytes % 4 == 0 &&
         ld <= (int64_t)0xFFFF0000u / 256 / bytes;
}

// GEMM_LP_TILE=<256|128|64|644> forces a tile where it has a kernel, for tests and measurement, as
// GEMMF32_VARIANT does for the FP32 product.
static int env_tile() {
  const char* v = std::getenv("GEMM_LP_TILE");
  return v == nullptr ? 0 : std::atoi(v);
}
// Time of one 128-byte K step of a tile, in us, measured on MI355X: `alone` with one workgroup
// on the CU, `full` a CU's time for each with as many as fit (and the chip as warm as it gets);
// a tile's own first loads and last stores cost it about `extra` steps, fewer where others fill
// the gap.  A CU works through n = ceil(tiles / 256) tiles in n * full or, where that is more,
// in rounds of `fit` tiles of `alone`; a launch adds about 4 us to all.
struct StepCost {
  double alone, full, extra;
};
constexpr int kFit[kTileCount] = {1, 2, 4, 1};
constexpr StepCost kStep16[kTileCount] = {
    {1.40, 1.75, 2}, {0.80, 0.60, 2}, {0.45, 0.24, 2}, {0.25, 0.25, 2}};
constexpr StepCost kStep16Grad[kTileCount] = {
    {1.40, 1.60, 5}, {0.80, 0.62, 2.8}, {0.45, 0.22, 2.4}, {0.25, 0.25, 10}};
constexpr StepCost kStep32[kTileCount] = {
    {7.30, 7.30, 2}, {2.00, 1.87, 3.5}, {0.66, 0.51, 0.7}, {0.60, 0.60, 2}};
constexpr StepCost kStep8[kTileCount] = {
    {0, 0, 0}, {1.20, 0.93, 2}, {0.60, 0.36, 2}, {0.37, 0.37, 2}};

// The tile of the pipelined kernels with the least time; `rounds(tile)` is the number of rounds
// of tiles on all CUs to expect, and the longest tile has `skew` times the average's K steps.
// rows: a row product.  Over 48 random sizes of every product and type the choice took 0 to 2 %
// longer on average than the best of all tiles, and at worst 1.35 times as long (a weight gradient
// of 8 rows in all; of those above 20 us 1.2 times).  Weight gradients of few experts are its weak
// spot: their longest expert decides, whose rows the host does not know, only `skew`.
constexpr int kForced[kTileCount] = {256, 128, 64, 644};
template <class F>
static int pick_tile(int unit, bool staged, bool rows, double steps, double skew, F rounds) {
  if (const int forced = env_tile()) {
    for (int t = 0; t < kTileCount; ++t)
      if (kForced[t] == forced && pipe_kernel(unit, t, staged) != nullptr) return t;
  }
  const StepCost* cost = unit < 6 ? (rows ? kStep16 : kStep16Grad)
                         : unit < 9 ? kStep32
                                    : kStep8;
  int best = -1;
  double least = 0;
  for (int t = 0; t < kTileCount; ++t) {
    if (pipe_kernel(unit, t, staged) == nullptr) continue;
    const double n = rounds(t);
    const double us = std::max({(steps + cost[t].extra) * n * cost[t].full,
                                (steps + cost[t].extra) * (n < 1 ? n : std::ceil(n / kFit[t])) *
                                    cost[t].alone,
                                (skew * steps + cost[t].extra) * cost[t].alone});
    if (best < 0 || us < least) best = t, least = us;
  }
  return best;
}

// Rounds of tiles on all CUs to expect of a row product: every group with rows leaves half a
// tile row unused (a quarter where the tile is computed in halves) and has one tile at least;
// one group alone has all rows.
static double row_rounds(const LpArgs& a, int unit, int tile) {
  const double bm = kTiles[tile].bm, half = half_cost(unit, tile);
  const double tn = std::ceil((double)a.N / kTiles[tile].bn), groups = std::min(a.E, a.rows);
  const bool many = a.offsets != nullptr && a.E > 1;
  if (many && half < 1 && a.rows <= groups * bm / 2)  // half tiles only
    return std::ceil(groups * tn / kCus) * half;
  const double m = !many ? std::ceil(a.rows / bm)
                         : std::max(a.rows / bm + (half < 1 ? 0.25 : 0.5) * groups, groups * half);
  const double n = m * tn / kCus, rest = n - std::floor(n);
  return std::floor(n) + (rest == 0 ? 0 : rest <= 0.5 ? half : 1);
}
static double k_steps(int64_t k, int bytes) { return std::ceil((double)k * bytes / kRowBytes); }

template <class T, bool EXP>
static const void* quantize_kernel(bool rows_only, int block_rows) {
  if (rows_only) return (const void*)&lp_quantize_rows_kernel<T, EXP>;
  return block_rows == 1 ? (const void*)&lp_quantize_tile_kernel<T, 1, EXP>
                         : (const void*)&lp_quantize_tile_kernel<T, kBlock, EXP>;
}
template <bool EXP>
static const void* quantize_kernel(int type, bool rows_only, int block_rows) {
  switch (type) {
    case GEMM_LP_BF16: return quantize_kernel<Bf16, EXP>(rows_only, block_rows);
    case GEMM_LP_F16: return quantize_kernel<F16, EXP>(rows_only, block_rows);
    default: return quantize_kernel<F32, EXP>(rows_only, block_rows);
  }
}

// EXP: scales as exponent bytes, [block][row]; otherwise FP32 numbers, [row block][block].
template <bool EXP>
static int run_quantize(int64_t rows, int64_t cols, const void* X, int64_t ldx, int type,
                        int block_rows, void* Q, int64_t ldq, void* S, int64_t lds, void* QT,
                        int64_t ldqt, void* ST, int64_t ldst, void* stream) {
  if (rows < 0 || cols < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (block_rows != 1 && block_rows != kBlock) return GEMMF32_ERR_BAD_CONFIG;
  if ((Q == nullptr) != (S == nullptr) || (QT == nullptr) != (ST == nullptr))
    return GEMMF32_ERR_NULL_PTR;
  const int64_t kb = blocks(cols), mb = blocks(rows);
  // rows and columns of the two arrays of scales, and the bytes of one
  const int64_t s_rows = EXP ? kb : block_rows == 1 ? rows : mb, s_cols = EXP ? rows : kb;
  const int64_t st_rows = EXP ? mb : block_rows == 1 ? cols : kb, st_cols = EXP ? cols : mb;
  constexpr int sb = EXP ? 1 : 4;
  if (ldx < at_least_1(cols) || (Q && (ldq < at_least_1(cols) || lds < at_least_1(s_cols))) ||
      (QT && (ldqt < at_least_1(rows) || ldst < at_least_1(st_cols))))
    return GEMMF32_ERR_BAD_LD;
  if (rows > kMaxDim || cols > kMaxDim) return GEMMF32_ERR_TOO_LARGE;
  if (rows == 0 || cols == 0) return GEMMF32_OK;
  if (X == nullptr || (Q == nullptr && QT == nullptr)) return GEMMF32_ERR_NULL_PTR;
  const int xb = type_bytes(type);
  if (misaligned(X, xb) || misaligned(S, sb) || misaligned(ST, sb))
    return GEMMF32_ERR_MISALIGNED;
  Range x, out[4];
  if (!byte_range(X, 1, 0, rows, cols, ldx, xb, &x)) return GEMMF32_ERR_TOO_LARGE;
  if (Q && (!byte_range(Q, 1, 0, rows, cols, ldq, 1, &out[0]) ||
            !byte_range(S, 1, 0, s_rows, s_cols, lds, sb, &out[1])))
    return GEMMF32_ERR_TOO_LARGE;
  if (QT && (!byte_range(QT, 1, 0, cols, rows, ldqt, 1, &out[2]) ||
             !byte_range(ST, 1, 0, st_rows, st_cols, ldst, sb, &out[3])))
    return GEMMF32_ERR_TOO_LARGE;
  for (int i = 0; i < 4; ++i) {
    if (overlap(out[i], x)) return GEMMF32_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return GEMMF32_ERR_ALIAS;
  }
  QuantArgs a{X,   (uint8_t*)Q, S,    (uint8_t*)QT, ST,       ldx,
              ldq, lds,         ldqt, ldst,         (int)rows, (int)cols};
  const bool rows_only = QT == nullptr && block_rows == 1;
  const void* fn = quantize_kernel<EXP>(type, rows_only, block_rows);
  if (rows_only) {
    const int64_t wgs = (rows * kb + 15) / 16;
    if (wgs > 0xFFFFFFFFLL / 256) return GEMMF32_ERR_TOO_LARGE;
    return launch(fn, dim3((unsigned)wgs), 256, &a, stream);
  }
  const int64_t wgs = mb * kb;  // (each at most 2^24)
  if (wgs > 0xFFFFFFFFLL / 256) return GEMMF32_ERR_TOO_LARGE;
  return launch(fn, dim3((unsigned)wgs), 256, &a, stream);
}

// EXP: the scales are exponent bytes, [block][row], as run_quantize writes them.
template <bool EXP>
static int run_fp8(int64_t M, int64_t N, int64_t K, int64_t E, const int32_t* offsets,
                   const void* A, int64_t lda, const void* SA, int64_t ldsa, const void* B,
                   int64_t ldb, int64_t stride_b, const void* SB, int64_t ldsb,
                   int64_t stride_sb, int b_block, void* C, int64_t ldc, int c_type,
                   void* stream) {
  if (M < 0 || N < 0 || K < 0 || E < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(c_type)) return GEMMF32_ERR_BAD_TYPE;
  if ((b_block != 1 && b_block != kBlock) || (offsets == nullptr && E != 1))
    return GEMMF32_ERR_BAD_CONFIG;
  const int64_t kb = blocks(K), nb = b_block == 1 ? N : blocks(N);
  const int64_t sa_rows = EXP ? kb : M, sa_cols = EXP ? M : kb;
  const int64_t sb_rows = EXP ? kb : nb, sb_cols = EXP ? N : kb;
  if (lda < at_least_1(K) || ldb < at_least_1(K) || ldc < at_least_1(N) ||
      ldsa < at_least_1(sa_cols) || ldsb < at_least_1(sb_cols) || stride_b < 0 || stride_sb < 0 ||
      (EXP && (ldsa % 4 != 0 || ldsb % 4 != 0)))
    return GEMMF32_ERR_BAD_LD;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim || E > kMaxDim ||
      (!EXP && (ldsa >= kMaxScaleLd || ldsb >= kMaxScaleLd)))
    return GEMMF32_ERR_TOO_LARGE;
  if (M == 0 || N == 0) return GEMMF32_OK;
  if (C == nullptr) return GEMMF32_ERR_NULL_PTR;
  const bool reads = K > 0 && E > 0;
  if (reads && (A == nullptr || B == nullptr || SA == nullptr || SB == nullptr))
    return GEMMF32_ERR_NULL_PTR;
  const int cb = type_bytes(c_type);
  if (misaligned(C, cb) || misaligned(offsets, 4) ||
      (reads && (misaligned(SA, 4) || misaligned(SB, 4))))
    return GEMMF32_ERR_MISALIGNED;
  Range c, in[5];
  if (!byte_range(C, 1, 0, M, N, ldc, cb, &c)) return GEMMF32_ERR_TOO_LARGE;
  if (reads && (!byte_range(A, 1, 0, M, K, lda, 1, &in[0]) ||
                !byte_range(SA, 1, 0, sa_rows, sa_cols, ldsa, EXP ? 1 : 4, &in[1]) ||
                !byte_range(B, E, stride_b, N, K, ldb, 1, &in[2]) ||
                !byte_range(SB, E, stride_sb, sb_rows, sb_cols, ldsb, EXP ? 1 : 4, &in[3])))
    return GEMMF32_ERR_TOO_LARGE;
  if (offsets && !byte_range(offsets, 1, 0, 1, E + 1, E + 1, 4, &in[4]))
    return GEMMF32_ERR_TOO_LARGE;
  for (const Range& r : in)
    if (overlap(c, r)) return GEMMF32_ERR_ALIAS;
  LpArgs a{};
  a.A = A, a.B = B, a.C = C, a.offsets = offsets;
  a.SA = (const float*)SA, a.SB = (const float*)SB;
  a.lda = lda, a.ldb = ldb, a.ldc = ldc, a.stride_b = stride_b;
  a.ldsa = ldsa, a.ldsb = ldsb, a.stride_sb = stride_sb;
  a.rows = a.M = (int)M, a.N = (int)N, a.K = (int)K, a.E = (int)E;
  a.sb_shift = b_block == 1 ? 0 : 7, a.c_type = c_type;
  const int unit = EXP ? 11 : b_block == 1 ? 9 : 10;
  const bool staged = !(word_rows(A, lda, 0, 1) && word_rows(B, ldb, stride_b, 1));
  const int t = pick_tile(unit, staged, true, k_steps(K, 1), 1.0,
                          [&](int tile) { return row_rounds(a, unit, tile); });
  return launch_rows(unit, t, staged, a, stream);
}

static int run_grouped(int64_t rows, int64_t N, int64_t K, int64_t E, const int32_t* offsets,
                       const void* X, int64_t ldx, const void* W, int64_t ldw,
                       int64_t stride_w, int transpose_w, void* Y, int64_t ldy, int type,
                       void* stream) {
  if (rows < 0 || N < 0 || K < 0 || E < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  const int64_t wr = transpose_w ? N : K, wc = transpose_w ? K : N;
  if (ldx < at_least_1(K) || ldw < at_least_1(wc) || ldy < at_least_1(N) || stride_w < 0)
    return GEMMF32_ERR_BAD_LD;
  if (rows > kMaxDim || N > kMaxDim || K > kMaxDim || E > kMaxDim) return GEMMF32_ERR_TOO_LARGE;
  if (rows == 0 || N == 0) return GEMMF32_OK;
  const bool reads = K > 0 && E > 0;
  if (Y == nullptr || offsets == nullptr || (reads && (X == nullptr || W == nullptr)))
    return GEMMF32_ERR_NULL_PTR;
  const int b = type_bytes(type);
  if (misaligned(Y, b) || misaligned(offsets, 4) || (reads && (misaligned(X, b) || misaligned(W, b))))
    return GEMMF32_ERR_MISALIGNED;
  Range y, in[3];
  if (!byte_range(Y, 1, 0, rows, N, ldy, b, &y) ||
      !byte_range(offsets, 1, 0, 1, E + 1, E + 1, 4, &in[2]) ||
      (reads && (!byte_range(X, 1, 0, rows, K, ldx, b, &in[0]) ||
                 !byte_range(W, E, stride_w, wr, wc, ldw, b, &in[1]))))
    return GEMMF32_ERR_TOO_LARGE;
  for (const Range& r : in)
    if (overlap(y, r)) return GEMMF32_ERR_ALIAS;
  LpArgs a{};
  a.A = X, a.B = W, a.C = Y, a.offsets = offsets;
  a.lda = ldx, a.ldb = ldw, a.ldc = ldy, a.stride_b = stride_w;
  a.rows = a.M = (int)rows, a.N = (int)N, a.K = (int)K, a.E = (int)E;
  a.c_type = type;
  const int unit = 3 * type + (transpose_w ? 0 : 1);
  const bool staged = !(word_rows(X, ldx, 0, b) && word_rows(W, ldw, stride_w, b));
  const int t = pick_tile(unit, staged, true, k_steps(K, b), 1.0,
                          [&](int tile) { return row_rounds(a, unit, tile); });
  return launch_rows(unit, t, staged, a, stream);
}

static int run_wgrad(int64_t rows, int64_t M, int64_t N, int64_t E, const int32_t* offsets,
                     const void* A, int64_t lda, const void* B, int64_t ldb, void* dW,
                     int64_t ldw, int64_t stride_w, int type, void* stream) {
  if (rows < 0 || M < 0 || N < 0 || E < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (lda < at_least_1(M) || ldb < at_least_1(N) || ldw < at_least_1(N)) return GEMMF32_ERR_BAD_LD;
  if (rows > kMaxDim || M > kMaxDim || N > kMaxDim || E > kMaxDim) return GEMMF32_ERR_TOO_LARGE;
  if (M == 0 || N == 0 || E == 0) return GEMMF32_OK;
  const bool reads = rows > 0;
  if (dW == nullptr || offsets == nullptr || (reads && (A == nullptr || B == nullptr)))
    return GEMMF32_ERR_NULL_PTR;
  const int b = type_bytes(type);
  if (misaligned(dW, b) || misaligned(offsets, 4) || (reads && (misaligned(A, b) || misaligned(B, b))))
    return GEMMF32_ERR_MISALIGNED;
  Range w, in[3], one;
  if (!byte_range(dW, E, stride_w, M, N, ldw, b, &w) ||
      !byte_range(dW, 1, 0, M, N, ldw, b, &one) ||
      !byte_range(offsets, 1, 0, 1, E + 1, E + 1, 4, &in[2]) ||
      (reads && (!byte_range(A, 1, 0, rows, M, lda, b, &in[0]) ||
                 !byte_range(B, 1, 0, rows, N, ldb, b, &in[1]))))
    return GEMMF32_ERR_TOO_LARGE;
  // each expert's dW has to end where the next begins, or it would be written twice
  if (E > 1 && (stride_w < 0 || (uint64_t)stride_w * b < (uint64_t)(one.hi - one.lo)))
    return GEMMF32_ERR_BAD_LD;
  for (const Range& r : in)
    if (overlap(w, r)) return GEMMF32_ERR_ALIAS;
  LpArgs a{};
  a.A = A, a.B = B, a.C = dW, a.offsets = offsets;
  a.lda = lda, a.ldb = ldb, a.ldc = ldw, a.stride_c = stride_w;
  a.rows = a.K = (int)rows, a.M = (int)M, a.N = (int)N, a.E = (int)E;
  a.c_type = type;
  const int unit = 3 * type + 2;
  const bool staged = !(word_rows(A, lda, 0, b) && word_rows(B, ldb, 0, b));
  // (the largest of four experts commonly has twice the average's rows, of 16 three times)
  const double skew = std::min(3.0, 1.0 + 0.5 * std::log2((double)E));
  const int t = pick_tile(unit, staged, false, k_steps((rows + E - 1) / E, b), skew, [&](int tile) {
    return std::ceil(std::ceil((double)M / kTiles[tile].bm) *
                     std::ceil((double)N / kTiles[tile].bn) * (double)E / kCus);
  });
  return launch_wgrad(unit, t, staged, a, stream);
}

}  // namespace gemmlp

extern "C" {

int gemm_fp8_quantize(int64_t rows, int64_t cols, const void* X, int64_t ldx, int type,
                      int block_rows, void* Q, int64_t ldq, float* S, int64_t lds, void* QT,
                      int64_t ldqt, float* ST, int64_t ldst, void* stream) {
  return gemmlp::run_quantize<false>(rows, cols, X, ldx, type, block_rows, Q, ldq, S, lds, QT,
                                     ldqt, ST, ldst, stream);
}

int gemm_fp8_quantize_exp(int64_t rows, int64_t cols, const void* X, int64_t ldx, int type,
                          int block_rows, void* Q, int64_t ldq, uint8_t* S, int64_t lds, void* QT,
                          int64_t ldqt, uint8_t* ST, int64_t ldst, void* stream) {
  return gemmlp::run_quantize<true>(rows, cols, X, ldx, type, block_rows, Q, ldq, S, lds, QT,
                                    ldqt, ST, ldst, stream);
}

int gemm_fp8(int64_t M, int64_t N, int64_t K, int64_t E, const int32_t* offsets, const void* A,
             int64_t lda, const float* SA, int64_t ldsa, const void* B, int64_t ldb,
             int64_t stride_b, const float* SB, int64_t ldsb, int64_t stride_sb, int b_block,
             void* C, int64_t ldc, int c_type, void* stream) {
  return gemmlp::run_fp8<false>(M, N, K, E, offsets, A, lda, SA, ldsa, B, ldb, stride_b, SB,
                                ldsb, stride_sb, b_block, C, ldc, c_type, stream);
}

int gemm_fp8_exp(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const uint8_t* SA,
                 int64_t ldsa, const void* B, int64_t ldb, const uint8_t* SB, int64_t ldsb,
                 void* C, int64_t ldc, int c_type, void* stream) {
  return gemmlp::run_fp8<true>(M, N, K, 1, nullptr, A, lda, SA, ldsa, B, ldb, 0, SB, ldsb, 0, 1,
                               C, ldc, c_type, stream);
}

int gemm_grouped(int64_t rows, int64_t N, int64_t K, int64_t E, const int32_t* offsets,
                 const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t stride_w,
                 int transpose_w, void* Y, int64_t ldy, int type, void* stream) {
  return gemmlp::run_grouped(rows, N, K, E, offsets, X, ldx, W, ldw, stride_w, transpose_w, Y,
                             ldy, type, stream);
}

int gemm_grouped_wgrad(int64_t rows, int64_t M, int64_t N, int64_t E, const int32_t* offsets,
                       const void* A, int64_t lda, const void* B, int64_t ldb, void* dW,
                       int64_t ldw, int64_t stride_w, int type, void* stream) {
  return gemmlp::run_wgrad(rows, M, N, E, offsets, A, lda, B, ldb, dW, ldw, stride_w, type,
                           stream);
}

}  // extern "C"
