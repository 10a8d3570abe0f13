/*
 * gemm_lp -- low-precision and expert-grouped matrix products for AMD MI355X (gfx950),
 * in the same library as gemmf32 and with its conventions.
 *
 * Operators
 *   gemm_fp8_quantize   values -> 8-bit floating point (OCP e4m3fn), one power-of-two scale
 *                       for each 1 x 128 or 128 x 128 block; optionally the transpose too
 *   gemm_fp8_quantize_exp  the same with the scales as exponent bytes
 *   gemm_fp8            C = (A sa)(B sb)^T for 8-bit A, B with a scale for each block of 128
 *                       along K; optionally one B per expert and ragged groups of rows
 *   gemm_fp8_exp        one such product with exponent bytes for scales
 *   gemm_grouped        Y[t] = X[t] W_e for the rows t of expert e, in bf16, fp16 or fp32
 *   gemm_grouped_wgrad  dW_e = sum over the rows t of expert e of A[t]^T B[t]
 *
 * Groups: `offsets` is a DEVICE array of E + 1 int32 with 0 <= offsets[0] <= ... <=
 * offsets[E] <= rows; rows offsets[e] .. offsets[e+1] - 1 belong to expert e, and the rows
 * before offsets[0] and from offsets[E] on belong to none: their results are zeros.  The
 * kernels read it, so no size has to come back to the host.  Its values cannot be checked
 * on the host; the kernels clamp each to [0, rows] and take a range that ends before it
 * begins as empty, so that wrong ones give undefined values but no access out of bounds.
 *
 * Conventions shared with gemmf32.h: caller-owned device pointers, asynchronous launches on
 * `stream` (NULL = the default stream), no allocation, no state between calls, arguments
 * validated before any HIP call, return 0 or a GEMMF32_ERR_* code.  An output that overlaps
 * an input is GEMMF32_ERR_ALIAS.  Sums are held in FP32 and rounded once at the end.
 */
#ifndef GEMM_LP_H
#define GEMM_LP_H

#include <stdint.h>

#include "gemmf32.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum {
    GEMM_LP_BF16 = 0,
    GEMM_LP_F16 = 1,
    GEMM_LP_F32 = 2
};

/* Q = round(X / s), S = s: the scale s of a block_rows x 128 block of X (block_rows 1 or
 * 128) is the smallest power of two, at least 2^-126, that brings the block's largest finite
 * magnitude to 448 or less; Inf and NaN become NaN and leave the scale alone.  X is
 * rows x cols of `type` with row stride ldx; Q is rows x cols bytes with row stride ldq, S
 * is ceil(rows / block_rows) x ceil(cols / 128) with row stride lds.
 * QT, ST (both or neither): the same for the transpose of X, cols x rows bytes with row
 * stride ldqt and ceil(cols / block_rows) x ceil(rows / 128) scales with row stride ldst.
 * Q, S may be NULL (both) where only the transpose is wanted.
 * GEMMF32_ERR_TOO_LARGE past 2^24 - 1 workgroups, of which each takes a block of 128 x 128, or
 * sixteen of 1 x 128 where only Q and S of such blocks are wanted. */
int gemm_fp8_quantize(int64_t rows, int64_t cols, const void *X, int64_t ldx, int type,
                      int block_rows, void *Q, int64_t ldq, float *S, int64_t lds,
                      void *QT, int64_t ldqt, float *ST, int64_t ldst, void *stream);

/* The same with the scales as bytes e + 127 (2^e the scale), one for each row of Q and block of
 * 128 columns, block by block: S is ceil(cols / 128) x rows with row stride lds, ST is
 * ceil(rows / 128) x cols with row stride ldst.  The rows of a 128 x 128 block have one value. */
int gemm_fp8_quantize_exp(int64_t rows, int64_t cols, const void *X, int64_t ldx, int type,
                          int block_rows, void *Q, int64_t ldq, uint8_t *S, int64_t lds,
                          void *QT, int64_t ldqt, uint8_t *ST, int64_t ldst, void *stream);

/* C[i][j] = sum_k A[i][k] sa[i][k/128] B[j][k] sb[j/b_block][k/128].
 * A: M x K e4m3fn, row stride lda; SA: M x ceil(K/128), row stride ldsa.
 * B: N x K e4m3fn, row stride ldb; SB: ceil(N/b_block) x ceil(K/128), row stride ldsb;
 * b_block is 1 or 128.  C: M x N of c_type, row stride ldc.  Any alignment of A and B.
 * sa and sb are any FP32 numbers, and their product is formed in FP32: where it overflows, so
 * does the block's part of C; where it falls below 2^-149 that part is lost.  ldsa and ldsb are
 * below 2^22.
 * offsets == NULL: one product (E must be 1).  Otherwise E experts: expert e's B and SB
 * start e * stride_b bytes and e * stride_sb floats after the first's, and rows of no
 * expert are zeroed in C. */
int gemm_fp8(int64_t M, int64_t N, int64_t K, int64_t E, const int32_t *offsets,
             const void *A, int64_t lda, const float *SA, int64_t ldsa,
             const void *B, int64_t ldb, int64_t stride_b,
             const float *SB, int64_t ldsb, int64_t stride_sb, int b_block,
             void *C, int64_t ldc, int c_type, void *stream);

/* gemm_fp8 of one product whose scales are gemm_fp8_quantize_exp's bytes: SA is ceil(K/128) x M,
 * SB ceil(K/128) x N, both 4-byte aligned with row strides that are multiples of 4. */
int gemm_fp8_exp(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const uint8_t *SA,
                 int64_t ldsa, const void *B, int64_t ldb, const uint8_t *SB, int64_t ldsb,
                 void *C, int64_t ldc, int c_type, void *stream);

/* Y (rows x N) = X (rows x K) W_e, all of `type`.  W_e starts e * stride_w elements after W:
 * K x N with row stride ldw, or with transpose_w N x K (Y = X W_e^T). */
int gemm_grouped(int64_t rows, int64_t N, int64_t K, int64_t E, const int32_t *offsets,
                 const void *X, int64_t ldx, const void *W, int64_t ldw, int64_t stride_w,
                 int transpose_w, void *Y, int64_t ldy, int type, void *stream);

/* dW_e (M x N, row stride ldw, e * stride_w elements after dW) = A_e^T B_e over the rows of
 * expert e: A is rows x M, B is rows x N, all of `type`.  An expert without rows gets zeros. */
int gemm_grouped_wgrad(int64_t rows, int64_t M, int64_t N, int64_t E, const int32_t *offsets,
                       const void *A, int64_t lda, const void *B, int64_t ldb,
                       void *dW, int64_t ldw, int64_t stride_w, int type, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* GEMM_LP_H */
