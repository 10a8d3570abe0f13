// Host side of the operators around the experts' products (but for the adapters): argument checks,
// the choice of a kernel, launches, and the C ABI of include/gemm_experts.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ex_gated.h"
#include "ex_group.h"
#include "ex_route.h"
#include "gemm_experts.h"
#include "lp_host.h"

namespace gemmlp {

// ---------------------------------------------------------------------------------- router
// Lanes of a row and logits of a lane: 16 lanes as long as each holds 16 logits or fewer, so that
// a wave's reductions serve four rows at once.
enum { kRoute16x1, kRoute16x4, kRoute16x16, kRoute64x16, kRouteKinds };
static int route_kind(int64_t E) {
  return E <= 16 ? kRoute16x1 : E <= 64 ? kRoute16x4 : E <= 256 ? kRoute16x16 : kRoute64x16;
}
static int64_t route_rows(int64_t E, int threads) { return threads / (E <= 256 ? 16 : 64); }
// Workgroups of the forward pass: one a CU at most, as their sums are added by one workgroup.
static int64_t route_groups(int64_t rows, int64_t E) {
  const int64_t per = route_rows(E, kRouteThreads);
  return std::min<int64_t>((rows + per - 1) / per, kCus);
}

template <class T>
static const void* route_kernel(int kind, bool grad) {
  switch (kind) {
    case kRoute16x1:
      return grad ? (const void*)&ex_route_grad_kernel<T, 16, 1> : (const void*)&ex_route_kernel<T, 16, 1>;
    case kRoute16x4:
      return grad ? (const void*)&ex_route_grad_kernel<T, 16, 4> : (const void*)&ex_route_kernel<T, 16, 4>;
    case kRoute16x16:
      return grad ? (const void*)&ex_route_grad_kernel<T, 16, 16> : (const void*)&ex_route_kernel<T, 16, 16>;
    default:
      return grad ? (const void*)&ex_route_grad_kernel<T, 64, 16> : (const void*)&ex_route_kernel<T, 64, 16>;
  }
}
static const void* route_kernel(int type, int kind, bool grad) {
  return type == GEMM_LP_BF16  ? route_kernel<Bf16>(kind, grad)
         : type == GEMM_LP_F16 ? route_kernel<F16>(kind, grad)
                               : route_kernel<F32>(kind, grad);
}

static int64_t route_workspace(int64_t rows, int64_t E) {
  const int64_t g = route_groups(rows, E);
  return g > 1 ? g * (2 * E + 1) * 4 : 0;
}
static int route_sizes(int64_t rows, int64_t E, int64_t k, int type) {
  if (rows < 0 || E < 0 || k < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (E < 1 || E > GEMM_ROUTE_MAX_EXPERTS || k < 1 || k > GEMM_ROUTE_MAX_CHOSEN || k > E)
    return GEMMF32_ERR_BAD_CONFIG;
  return GEMMF32_OK;
}

static int run_route(int64_t rows, int64_t E, int64_t k, const void* X, int64_t ldx, int type,
                     const uint8_t* valid, int renormalize, float* gates, int32_t* experts,
                     int32_t* counts, int32_t* sums, float* loss, void* workspace,
                     int64_t workspace_bytes, void* stream) {
  if (const int rc = route_sizes(rows, E, k, type)) return rc;
  const int64_t need = route_workspace(rows, E);
  if (ldx < E || workspace_bytes < need) return GEMMF32_ERR_BAD_LD;
  if (rows > kMaxDim / k) return GEMMF32_ERR_TOO_LARGE;  // (counts and their sum are 32-bit)
  if (counts == nullptr || sums == nullptr || loss == nullptr || (need && workspace == nullptr) ||
      (rows && (X == nullptr || gates == nullptr || experts == nullptr)))
    return GEMMF32_ERR_NULL_PTR;
  if (misaligned(X, type_bytes(type)) || misaligned(gates, 4) || misaligned(experts, 4) ||
      misaligned(counts, 4) || misaligned(sums, 4) || misaligned(loss, 4) ||
      misaligned(workspace, 8))
    return GEMMF32_ERR_MISALIGNED;
  Range out[6], in[2];
  if ((rows && (!byte_range(X, 1, 0, rows, E, ldx, type_bytes(type), &in[0]) ||
                !row_range(gates, rows * k, 4, &out[0]) || !row_range(experts, rows * k, 4, &out[1]))) ||
      (rows && valid && !row_range(valid, rows, 1, &in[1])) || !row_range(counts, E, 4, &out[2]) ||
      !row_range(sums, 2, 4, &out[3]) || !row_range(loss, 1, 4, &out[4]) ||
      (need && !row_range(workspace, need, 1, &out[5])))
    return GEMMF32_ERR_TOO_LARGE;
  if (any_overlap(out, in)) return GEMMF32_ERR_ALIAS;
  RouteArgs a{};
  a.X = X, a.valid = valid, a.gates = gates, a.experts = experts, a.counts = counts;
  a.sums = sums, a.loss = loss, a.ldx = ldx;
  a.rows = (int)rows, a.E = (int)E, a.k = (int)k, a.norm = renormalize != 0;
  a.groups = (int)std::max<int64_t>(route_groups(rows, E), 1);
  a.part_p = (float*)workspace;
  a.part_n = (int32_t*)(a.part_p + (int64_t)a.groups * E);
  if (const int rc = launch(route_kernel(type, route_kind(E), false), dim3(a.groups), kRouteThreads,
                            &a, stream))
    return rc;
  if (a.groups == 1) return GEMMF32_OK;
  return launch((const void*)&ex_route_finish_kernel, dim3(1), kRouteThreads, &a, stream);
}

static int run_route_grad(int64_t rows, int64_t E, int64_t k, const void* X, int64_t ldx, int type,
                          const uint8_t* valid, int renormalize, const float* gates,
                          const int32_t* experts, const int32_t* counts, const int32_t* sums,
                          const float* dgates, const float* dloss, void* DX, int64_t lddx,
                          void* stream) {
  if (const int rc = route_sizes(rows, E, k, type)) return rc;
  if (ldx < E || lddx < E) return GEMMF32_ERR_BAD_LD;
  if (rows > kMaxDim / k) return GEMMF32_ERR_TOO_LARGE;
  if (rows == 0) return GEMMF32_OK;
  if (X == nullptr || DX == nullptr || counts == nullptr || sums == nullptr ||
      (dgates && (gates == nullptr || experts == nullptr)))
    return GEMMF32_ERR_NULL_PTR;
  const int b = type_bytes(type);
  if (misaligned(X, b) || misaligned(DX, b) || misaligned(gates, 4) || misaligned(experts, 4) ||
      misaligned(counts, 4) || misaligned(sums, 4) || misaligned(dgates, 4) || misaligned(dloss, 4))
    return GEMMF32_ERR_MISALIGNED;
  Range out[1], in[8];
  if (!byte_range(DX, 1, 0, rows, E, lddx, b, &out[0]) ||
      !byte_range(X, 1, 0, rows, E, ldx, b, &in[0]) ||
      (valid && !row_range(valid, rows, 1, &in[1])) ||
      (dgates && (!row_range(gates, rows * k, 4, &in[2]) || !row_range(experts, rows * k, 4, &in[3]) ||
                  !row_range(dgates, rows * k, 4, &in[4]))) ||
      !row_range(counts, E, 4, &in[5]) || !row_range(sums, 2, 4, &in[6]) ||
      (dloss && !row_range(dloss, 1, 4, &in[7])))
    return GEMMF32_ERR_TOO_LARGE;
  if (any_overlap(out, in)) return GEMMF32_ERR_ALIAS;
  RouteArgs a{};
  a.X = X, a.valid = valid, a.gates = (float*)gates, a.experts = (int32_t*)experts;
  a.counts = (int32_t*)counts, a.sums = (int32_t*)sums, a.dgates = dgates, a.dloss = dloss;
  a.DX = DX, a.ldx = ldx, a.lddx = lddx;
  a.rows = (int)rows, a.E = (int)E, a.k = (int)k, a.norm = renormalize != 0;
  const int64_t per = route_rows(E, kRouteGradThreads);
  const int64_t groups = std::min<int64_t>((rows + per - 1) / per, 16 * kCus);
  return launch(route_kernel(type, route_kind(E), true), dim3((unsigned)groups), kRouteGradThreads,
                &a, stream);
}

// --------------------------------------------------------------------------------- grouping
// Rows of a workgroup, a multiple of 64 for each of its waves: one workgroup alone up to
// kGroupAlone rows, which saves a launch (2048 rows of 64 experts 5.8 us either way, 4096 9.1 and 5.7,
// 8192 16 and 5.8); from there on 2048 each or fewer, and more where there would be more than 128
// workgroups, each of which reads the counts of all.  There are sixteens of them, of which the last may
// have no rows: the counts are read 16 at a time, and what is left of a 16 one by one (20000 rows 7.6
// us, 11 with ten workgroups; 60000 of 256 experts 10.5, 13 with 30).
constexpr int64_t kGroupAlone = 2048;
static int64_t up_to(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }
static int64_t group_run(int64_t n) {
  if (n <= kGroupAlone) return std::max<int64_t>(up_to(n, kGroupThreads), kGroupThreads);
  const int64_t workgroups = std::min<int64_t>(up_to((n + 2047) / 2048, 16), 128);
  return up_to((n + workgroups - 1) / workgroups, kGroupThreads);
}
static int64_t group_workgroups(int64_t n) {
  return n <= kGroupAlone ? 1 : up_to((n + group_run(n) - 1) / group_run(n), 16);
}
static int64_t group_workspace(int64_t n, int64_t E) {
  const int64_t g = group_workgroups(n);
  return g > 1 ? g * (E + 1) * 4 : 0;
}

static int run_group(int64_t n, int64_t E, const void* ids, int id_bytes, int64_t* order,
                     int64_t* place, int32_t* offsets, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  if (n < 0 || E < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (id_bytes != 4 && id_bytes != 8) return GEMMF32_ERR_BAD_TYPE;
  if (E > GEMM_GROUP_MAX_EXPERTS) return GEMMF32_ERR_BAD_CONFIG;
  if (n > kMaxDim) return GEMMF32_ERR_TOO_LARGE;
  const int64_t need = group_workspace(n, E);
  if (workspace_bytes < need) return GEMMF32_ERR_BAD_LD;
  if (offsets == nullptr || (need && workspace == nullptr) ||
      (n && (ids == nullptr || order == nullptr || place == nullptr)))
    return GEMMF32_ERR_NULL_PTR;
  if (misaligned(ids, id_bytes) || misaligned(order, 8) || misaligned(place, 8) ||
      misaligned(offsets, 4) || misaligned(workspace, 8))
    return GEMMF32_ERR_MISALIGNED;
  Range out[4], in[1];
  if ((n && (!row_range(ids, n, id_bytes, &in[0]) || !row_range(order, n, 8, &out[0]) ||
             !row_range(place, n, 8, &out[1]))) ||
      !row_range(offsets, E + 1, 4, &out[2]) || (need && !row_range(workspace, need, 1, &out[3])))
    return GEMMF32_ERR_TOO_LARGE;
  if (any_overlap(out, in)) return GEMMF32_ERR_ALIAS;
  GroupArgs a{ids, order, place, offsets, (int32_t*)workspace, (int)n, (int)E, id_bytes,
              (int)group_run(n), 0};
  while ((E >> a.bits) > 0) ++a.bits;
  const dim3 grid((unsigned)group_workgroups(n));
  const bool few = E <= 1024;
  if (grid.x > 1) {
    const void* fn = few ? (const void*)&ex_group_count_kernel<1024>
                         : (const void*)&ex_group_count_kernel<GEMM_GROUP_MAX_EXPERTS>;
    if (const int rc = launch(fn, grid, kGroupThreads, &a, stream)) return rc;
  }
  const void* fn = few ? (const void*)&ex_group_place_kernel<1024>
                       : (const void*)&ex_group_place_kernel<GEMM_GROUP_MAX_EXPERTS>;
  return launch(fn, grid, kGroupThreads, &a, stream);
}

// ------------------------------------------------------------------------------- gated unit
// Workgroups that hold 16 blocks of 128 columns each; 0 where there are too many.
static unsigned block_groups(int64_t rows, int64_t cols) {
  const int64_t n = (rows * blocks(cols) + 15) / 16;
  return n > 0xFFFFFFFFLL / 256 ? 0 : (unsigned)n;
}

template <class T>
static const void* gated_kernel(bool keep, bool grad) {
  if (grad)
    return keep ? (const void*)&ex_gated_grad_kernel<T, true> : (const void*)&ex_gated_grad_kernel<T, false>;
  return keep ? (const void*)&ex_gated_kernel<T, true> : (const void*)&ex_gated_kernel<T, false>;
}
static const void* gated_kernel(int type, bool keep, bool grad) {
  return type == GEMM_LP_BF16  ? gated_kernel<Bf16>(keep, grad)
         : type == GEMM_LP_F16 ? gated_kernel<F16>(keep, grad)
                               : gated_kernel<F32>(keep, grad);
}

// The forward pass where H is given, the gradient where DX is.
static int run_gated(int64_t rows, int64_t N, const void* X, int64_t ldx, void* Q, int64_t ldq,
                     float* S, int64_t lds, bool grad, const void* DH, int64_t lddh, void* out_rows,
                     int64_t ldout, int type, void* stream) {
  if (rows < 0 || N < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if ((Q == nullptr) != (S == nullptr)) return GEMMF32_ERR_NULL_PTR;
  if (rows > kMaxDim || N > kMaxDim / 2) return GEMMF32_ERR_TOO_LARGE;
  const int64_t sb = 2 * blocks(N);
  const bool reads_x = !grad || X != nullptr, keeps = Q != nullptr && !(grad && X != nullptr);
  if ((reads_x && ldx < at_least_1(2 * N)) ||
      (keeps && (ldq < at_least_1(2 * N) || lds < at_least_1(sb))) ||
      (grad && lddh < at_least_1(N)) || ldout < at_least_1(grad ? 2 * N : N))
    return GEMMF32_ERR_BAD_LD;
  if (rows == 0 || N == 0) return GEMMF32_OK;
  if ((reads_x ? X == nullptr : Q == nullptr) || out_rows == nullptr || (grad && DH == nullptr))
    return GEMMF32_ERR_NULL_PTR;
  const int b = type_bytes(type);
  if (misaligned(X, b) || misaligned(DH, b) || misaligned(out_rows, b) || misaligned(S, 4))
    return GEMMF32_ERR_MISALIGNED;
  Range x, dh, q, s, o;
  if ((reads_x && !byte_range(X, 1, 0, rows, 2 * N, ldx, b, &x)) ||
      (grad && !byte_range(DH, 1, 0, rows, N, lddh, b, &dh)) ||
      (keeps && (!byte_range(Q, 1, 0, rows, 2 * N, ldq, 1, &q) ||
                 !byte_range(S, 1, 0, rows, sb, lds, 4, &s))) ||
      !byte_range(out_rows, 1, 0, rows, grad ? 2 * N : N, ldout, b, &o))
    return GEMMF32_ERR_TOO_LARGE;
  if (grad ? any_overlap<1, 4>({o}, {x, dh, q, s}) : any_overlap<3, 1>({o, q, s}, {x}))
    return GEMMF32_ERR_ALIAS;
  const unsigned groups = block_groups(rows, N);
  if (groups == 0) return GEMMF32_ERR_TOO_LARGE;
  GatedArgs a{};
  a.X = X, a.Q = (uint8_t*)Q, a.S = S, a.DH = DH;
  a.ldx = ldx, a.ldq = ldq, a.lds = lds, a.lddh = lddh, a.rows = (int)rows, a.N = (int)N;
  if (grad) a.DX = out_rows, a.lddx = ldout;
  else a.H = out_rows, a.ldh = ldout;
  return launch(gated_kernel(type, keeps, grad), dim3(groups), 256, &a, stream);
}

static int run_dequantize(int64_t rows, int64_t cols, const void* Q, int64_t ldq, const float* S,
                          int64_t lds, int block_rows, void* Y, int64_t ldy, int type,
                          void* stream) {
  if (rows < 0 || cols < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (!known_type(type)) return GEMMF32_ERR_BAD_TYPE;
  if (block_rows != 1 && block_rows != kBlock) return GEMMF32_ERR_BAD_CONFIG;
  if (ldq < at_least_1(cols) || lds < at_least_1(blocks(cols)) || ldy < at_least_1(cols))
    return GEMMF32_ERR_BAD_LD;
  if (rows > kMaxDim || cols > kMaxDim) return GEMMF32_ERR_TOO_LARGE;
  if (rows == 0 || cols == 0) return GEMMF32_OK;
  if (Q == nullptr || S == nullptr || Y == nullptr) return GEMMF32_ERR_NULL_PTR;
  const int b = type_bytes(type);
  if (misaligned(Y, b) || misaligned(S, 4)) return GEMMF32_ERR_MISALIGNED;
  Range out[1], in[2];
  if (!byte_range(Q, 1, 0, rows, cols, ldq, 1, &in[0]) ||
      !byte_range(S, 1, 0, block_rows == 1 ? rows : blocks(rows), blocks(cols), lds, 4, &in[1]) ||
      !byte_range(Y, 1, 0, rows, cols, ldy, b, &out[0]))
    return GEMMF32_ERR_TOO_LARGE;
  if (any_overlap(out, in)) return GEMMF32_ERR_ALIAS;
  const unsigned groups = block_groups(rows, cols);
  if (groups == 0) return GEMMF32_ERR_TOO_LARGE;
  DequantArgs a{(const uint8_t*)Q, S, Y, ldq, lds, ldy, (int)rows, (int)cols,
                block_rows == 1 ? 0 : 7};
  const void* fn = type == GEMM_LP_BF16  ? (const void*)&ex_dequantize_kernel<Bf16>
                   : type == GEMM_LP_F16 ? (const void*)&ex_dequantize_kernel<F16>
                                         : (const void*)&ex_dequantize_kernel<F32>;
  return launch(fn, dim3(groups), 256, &a, stream);
}

}  // namespace gemmlp

extern "C" {

int gemm_route(int64_t rows, int64_t E, int64_t k, const void* X, int64_t ldx, int type,
               const uint8_t* valid, int renormalize, float* gates, int32_t* experts,
               int32_t* counts, int32_t* sums, float* loss, void* workspace,
               int64_t workspace_bytes, void* stream) {
  return gemmlp::run_route(rows, E, k, X, ldx, type, valid, renormalize, gates, experts, counts,
                           sums, loss, workspace, workspace_bytes, stream);
}

int64_t gemm_route_workspace(int64_t rows, int64_t E) {
  if (rows < 0 || E < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (rows > gemmlp::kMaxDim) return GEMMF32_ERR_TOO_LARGE;
  if (E > GEMM_ROUTE_MAX_EXPERTS) return GEMMF32_ERR_BAD_CONFIG;
  return gemmlp::route_workspace(rows, E);
}

int gemm_route_grad(int64_t rows, int64_t E, int64_t k, const void* X, int64_t ldx, int type,
                    const uint8_t* valid, int renormalize, const float* gates,
                    const int32_t* experts, const int32_t* counts, const int32_t* sums,
                    const float* dgates, const float* dloss, void* DX, int64_t lddx,
                    void* stream) {
  return gemmlp::run_route_grad(rows, E, k, X, ldx, type, valid, renormalize, gates, experts,
                                counts, sums, dgates, dloss, DX, lddx, stream);
}

int gemm_group_rows(int64_t n, int64_t E, const void* ids, int id_bytes, int64_t* order,
                    int64_t* place, int32_t* offsets, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  return gemmlp::run_group(n, E, ids, id_bytes, order, place, offsets, workspace, workspace_bytes,
                           stream);
}

int64_t gemm_group_rows_workspace(int64_t n, int64_t E) {
  if (n < 0 || E < 0) return GEMMF32_ERR_NEGATIVE_DIM;
  if (n > gemmlp::kMaxDim) return GEMMF32_ERR_TOO_LARGE;
  if (E > GEMM_GROUP_MAX_EXPERTS) return GEMMF32_ERR_BAD_CONFIG;
  return gemmlp::group_workspace(n, E);
}

int gemm_gated(int64_t rows, int64_t N, const void* X, int64_t ldx, int type, void* H, int64_t ldh,
               void* Q, int64_t ldq, float* S, int64_t lds, void* stream) {
  return gemmlp::run_gated(rows, N, X, ldx, Q, ldq, S, lds, false, nullptr, 0, H, ldh, type,
                           stream);
}

int gemm_gated_grad(int64_t rows, int64_t N, const void* X, int64_t ldx, const void* Q, int64_t ldq,
                    const float* S, int64_t lds, const void* DH, int64_t lddh, void* DX,
                    int64_t lddx, int type, void* stream) {
  return gemmlp::run_gated(rows, N, X, ldx, (void*)Q, ldq, (float*)S, lds, true, DH, lddh, DX,
                           lddx, type, stream);
}

int gemm_fp8_dequantize(int64_t rows, int64_t cols, const void* Q, int64_t ldq, const float* S,
                        int64_t lds, int block_rows, void* Y, int64_t ldy, int type,
                        void* stream) {
  return gemmlp::run_dequantize(rows, cols, Q, ldq, S, lds, block_rows, Y, ldy, type, stream);
}

}  // extern "C"
