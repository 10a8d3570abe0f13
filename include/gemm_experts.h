/*
 * gemm_experts -- what a layer of experts needs around its products, for AMD MI355X (gfx950),
 * in the same library as gemmf32 and gemm_lp and with their conventions.
 *
 * Operators
 *   gemm_route           softmax over experts, the k best of each row, rows of each expert, and the
 *                        balance loss; gemm_route_grad the gradient of the logits
 *   gemm_group_rows      rows in the order of their experts, and where each expert's begin
 *   gemm_adapters_*      out = y + s_e (x A_e^T) B_e, an adapter of low rank for each group of rows,
 *                        and its gradients
 *   gemm_gated           silu(gate) * up, optionally with both kept in 8 bits; gemm_gated_grad its
 *                        gradient from these values, or from the input
 *   gemm_fp8_dequantize  8-bit values with scales -> values
 *
 * Conventions shared with gemm_lp.h: caller-owned device pointers, asynchronous launches on
 * `stream` (NULL = the default stream), no allocation, no state between calls, arguments validated
 * before any HIP call, return 0 or a GEMMF32_ERR_* code, element types GEMM_LP_*.  An output that
 * overlaps an input or another output is GEMMF32_ERR_ALIAS.  No atomics whose order changes results:
 * the same call gives the same bits.
 */
#ifndef GEMM_EXPERTS_H
#define GEMM_EXPERTS_H

#include <stdint.h>

#include "gemm_lp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_ROUTE_MAX_EXPERTS 1024
#define GEMM_ROUTE_MAX_CHOSEN 16
#define GEMM_GROUP_MAX_EXPERTS 4096
#define GEMM_ADAPTERS_MAX_RANK 128
#define GEMM_ADAPTERS_MAX_SPLITS 64

/* The router of `rows` rows.  X: rows x E logits of `type`, row stride ldx.  valid: rows bytes, 0
 * for a row to be left out, or NULL.  A row counts if it is valid and has a logit above -Inf.
 *   p[t] = softmax(X[t]) of a row that counts
 *   experts[t][j], j < k: the j-th largest logit, of equal ones the lowest index; -1 where no logit
 *     above -Inf is left, and in rows that do not count
 *   gates[t][j] = p[t][experts[t][j]], with `renormalize` over the sum of the row's; 0 beside -1
 *   counts[e]: how often e was taken;  sums[0]: rows that count, sums[1]: the total of counts
 *   loss = E sum_e (counts[e] / sums[1]) (sum_t p[t][e] / sums[0]); 0 where no row counts
 * A NaN is taken before every number; it, or +Inf, makes its row's gates and the loss NaN.
 * Probabilities below 2^-126 may count as 0.
 * E <= GEMM_ROUTE_MAX_EXPERTS and k <= GEMM_ROUTE_MAX_CHOSEN, else GEMMF32_ERR_BAD_CONFIG, as for
 * k < 1 or k > E; rows k below 2^31 - 1024, else GEMMF32_ERR_TOO_LARGE.  workspace:
 * gemm_route_workspace(rows, E) bytes, 8-byte aligned (less is GEMMF32_ERR_BAD_LD; where that is 0 it
 * may be NULL); calls that overlap in time need one each. */
int gemm_route(int64_t rows, int64_t E, int64_t k, const void *X, int64_t ldx, int type,
               const uint8_t *valid, int renormalize, float *gates, int32_t *experts,
               int32_t *counts, int32_t *sums, float *loss, void *workspace,
               int64_t workspace_bytes, void *stream);
int64_t gemm_route_workspace(int64_t rows, int64_t E);

/* DX (rows x E of `type`, row stride lddx): the gradient of sum dgates gates + dloss loss in X,
 * counts as constants.  dgates: rows x k; dloss: one number on the device; either may be NULL (0).
 * gates, experts, counts, sums: gemm_route's results.  Rows that do not count get zeros. */
int gemm_route_grad(int64_t rows, int64_t E, int64_t k, const void *X, int64_t ldx, int type,
                    const uint8_t *valid, int renormalize, const float *gates,
                    const int32_t *experts, const int32_t *counts, const int32_t *sums,
                    const float *dgates, const float *dloss, void *DX, int64_t lddx,
                    void *stream);

/* Sorts n rows by expert, stably.  ids: n numbers of id_bytes (4 or 8) bytes; those outside
 * 0 .. E - 1 belong to no expert and come last.  order[i]: the row at place i; place[r]: the
 * place of row r; offsets[e], e <= E: the first place of expert e (of the rows of none).
 * E <= GEMM_GROUP_MAX_EXPERTS, else GEMMF32_ERR_BAD_CONFIG.  workspace:
 * gemm_group_rows_workspace(n, E) bytes, as in gemm_route. */
int gemm_group_rows(int64_t n, int64_t E, const void *ids, int id_bytes, int64_t *order,
                    int64_t *place, int32_t *offsets, void *workspace, int64_t workspace_bytes,
                    void *stream);
int64_t gemm_group_rows_workspace(int64_t n, int64_t E);

/* Adapters: expert (request, adapter) e has A_e, rank x K, and B_e, rank x N, `stride` elements
 * from one to the next, with unit column stride.  Places offsets[e] .. offsets[e+1] - 1 of `order`
 * hold its rows (offsets as in gemm_lp.h; order: `rows` int64 on the device, each row once; the
 * kernels clamp its values to 0 .. rows - 1, so that wrong ones give undefined values but no access
 * out of bounds).  rank <= GEMM_ADAPTERS_MAX_RANK and 1 <= splits <= GEMM_ADAPTERS_MAX_SPLITS, else
 * GEMMF32_ERR_BAD_CONFIG.
 *
 * down: U[p] = scale[e] X[order[p]] A_e^T for the places p of e, in FP32, as `splits` partial sums
 *   over K, each rows x 16 ceil(rank / 16) with zeros past the rank, one after another and 16-byte
 *   aligned (places of no expert are left as they were).  scale may be NULL (1).  With `join` the
 *   first holds their sum in the end (of places of no expert what it may), so that `up` and `grad`
 *   take it as one split: for many rows (about 1024 and more), as they read U several times.
 * up: OUT[order[p]] = Y[order[p]] + (sum of U's splits)[p] B_e; places of no expert: Y alone.
 *   Y may be NULL (0).
 * grad: DA_e (rank x K, row stride ldda, stride_da elements apart) = sum over the places p of e of
 *   V[p]^T X[order[p]], and DB_e (rank x N) = the same of U[p]^T DOUT[order[p]]; an expert without
 *   rows gets zeros.  Where only one is wanted the other's K or N is 0 (and its other arguments are
 *   not looked at).
 * Inf and NaN stay in their places' rows and their adapters.  In bf16 `up` and `grad` multiply U and V
 *   in three parts, of which one may be 0: Inf in A or B, and for grad in X or DOUT, gives NaN where
 *   the product is Inf; and of a U or V the bits below 2^-133, bf16's smallest step, are lost.
 * gemm_adapters_splits: the number of splits that `down` should make, at least 1.
 * gemm_adapters_grad_workspace: bytes of workspace that `grad` needs, as in gemm_route. */
int gemm_adapters_down(int64_t rows, int64_t K, int64_t rank, int64_t E, const int64_t *order,
                       const int32_t *offsets, const void *X, int64_t ldx, const void *A,
                       int64_t lda, int64_t stride_a, const float *scale, float *U, int splits,
                       int join, int type, void *stream);
int gemm_adapters_up(int64_t rows, int64_t N, int64_t rank, int64_t E, const int64_t *order,
                     const int32_t *offsets, const float *U, int splits, const void *B,
                     int64_t ldb, int64_t stride_b, const void *Y, int64_t ldy, void *OUT,
                     int64_t ldo, int type, void *stream);
int gemm_adapters_grad(int64_t rows, int64_t rank, int64_t E, const int64_t *order,
                       const int32_t *offsets, int64_t K, const float *V, int v_splits,
                       const void *X, int64_t ldx, void *DA, int64_t ldda, int64_t stride_da,
                       int64_t N, const float *U, int u_splits, const void *DOUT, int64_t ldd,
                       void *DB, int64_t lddb, int64_t stride_db, void *workspace,
                       int64_t workspace_bytes, int type, void *stream);
int gemm_adapters_splits(int64_t rows, int64_t K, int64_t rank, int64_t E);
int64_t gemm_adapters_grad_workspace(int64_t rows, int64_t K, int64_t N, int64_t rank, int64_t E,
                                     int type);

/* H = silu(G) * U, silu(g) = g / (1 + exp(-g)): X is rows x 2N, G its first N columns and U the
 * others; H rows x N.  Q, S (both or neither): G and U in 8 bits as gemm_fp8_quantize gives them,
 * each half by blocks of 1 x 128 of its own: Q rows x 2N bytes, row stride ldq; S rows x
 * 2 ceil(N / 128), row stride lds. */
int gemm_gated(int64_t rows, int64_t N, const void *X, int64_t ldx, int type, void *H, int64_t ldh,
               void *Q, int64_t ldq, float *S, int64_t lds, void *stream);

/* DX (rows x 2N) = (DH U silu'(G), DH silu(G)), with G and U from X, or where X is NULL from Q and
 * S (finite products past the type's range count as its largest number). */
int gemm_gated_grad(int64_t rows, int64_t N, const void *X, int64_t ldx, const void *Q, int64_t ldq,
                    const float *S, int64_t lds, const void *DH, int64_t lddh, void *DX,
                    int64_t lddx, int type, void *stream);

/* Y = Q S, Q rows x cols e4m3fn with one scale for each block_rows x 128 block (block_rows 1 or
 * 128), as gemm_fp8_quantize lays them out.  The product is formed in FP32, which rounds it unless S
 * is a power of two, as gemm_fp8_quantize's are, and is then rounded to `type`.  Finite products past
 * the type's range become its largest number. */
int gemm_fp8_dequantize(int64_t rows, int64_t cols, const void *Q, int64_t ldq, const float *S,
                        int64_t lds, int block_rows, void *Y, int64_t ldy, int type, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* GEMM_EXPERTS_H */
