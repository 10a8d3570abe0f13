// The router: softmax over the experts of a row, its k largest logits, the rows of each expert, and
// the balance loss
//   loss = E sum_e f_e P_e,  f_e = counts_e / sum counts,  P_e = sum_t p_te / n,
// n the rows that count; and the gradient of the logits.
//
// L lanes (16, or 64) share a row and hold V logits each; a row is read once, and its largest, the
// sum of exponentials and the k best come from the registers.  The k best are k searches for the
// largest order-preserving integer of the logit, then for the lowest index that has it.  A
// workgroup adds the probabilities of its rows in registers and counts in LDS (integers, whose
// order does not matter); the sums of all workgroups are added by one more launch, in a fixed
// order, or by the same workgroup where it is the only one.
//
// 16384 rows of 256 experts in FP32, k = 8: 16 us (16.8 MB; four rows a wave, whose eight searches of
// 40 instructions and 16 exponentials are most of it), 8.4 for the sums of 256 workgroups (half a
// megabyte that one CU reads), 20 for the gradient (33.5 MB, 6.8 us of a copy; its counts are loaded one
// after another before a row is).  16 rows of 64 experts, k = 4: 5.1 us.  A call
// takes the host 14 us, a step 100, of which autograd's own 37 are for a function that does nothing.
#pragma once

#include "ex_common.h"

namespace gemmlp {

struct RouteArgs {
  const void* X;
  const uint8_t* valid;
  float* gates;
  int32_t* experts;
  int32_t* counts;
  int32_t* sums;
  float* loss;
  float* part_p;     // [workgroup][E]: sums of probabilities
  int32_t* part_n;   // [workgroup][E + 1]: counts, and the rows that count
  const float* dgates;
  const float* dloss;
  void* DX;
  int64_t ldx, lddx;
  int rows, E, k, norm;
  int groups;        // workgroups whose sums there are
};

constexpr int kRouteThreads = 1024;
constexpr uint32_t kKeyNoExpert = 0x007fffffu;  // the key of -Inf

// Integers in the order of the numbers, NaN above all; both zeros have one.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  if (x != x) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Which columns a lane holds: groups of four neighbours, so that its loads are wide.
template <int L, int V>
__device__ __forceinline__ int column(int lane, int v) {
  if constexpr (V == 1) return lane;
  return ((v / 4) * L + lane) * 4 + v % 4;
}
// A lane's logits of a row, -Inf past the last: wide loads where groups of four end with the row.
template <class T, int L, int V>
__device__ __forceinline__ void load_logits(const void* X, int64_t at, int E, int lane, float* x) {
  const typename T::type* row = (const typename T::type*)X + at;
  const bool wide = V > 1 && E % 4 == 0;
  if constexpr (V > 1) {
    if (wide) {
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        const Raw<T, 4> r = load_raw<T, 4>(row + min(column<L, V>(lane, q), E - 4));
        x[q] = (float)r[0], x[q + 1] = (float)r[1], x[q + 2] = (float)r[2], x[q + 3] = (float)r[3];
      }
    }
  }
  if (!wide) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = (float)row[min(column<L, V>(lane, v), E - 1)];
  }
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = column<L, V>(lane, v) < E ? x[v] : -__builtin_inff();
}

// exp(x) for x <= 0 (and NaN), to 2^-22 of it: 2^(x log2 e), the product to 48 bits, as its rounding
// would count |x| times.  Below the smallest normal number it may be 0.
__device__ __forceinline__ float exp_below(float x) {
  constexpr float hi = 1.44269502e+00f, lo = 1.92596303e-08f;  // log2 e = hi + lo
  const float y = fmaxf(x, -1000.0f) * hi;
  const float rest = fmaf(fmaxf(x, -1000.0f), lo, fmaf(fmaxf(x, -1000.0f), hi, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return x == x ? fmaf(e * rest, 0.693147181f, e) : x;
}

// x becomes its softmax's numerators, over the largest; returns one over their sum.
template <int L, int V>
__device__ __forceinline__ float exponentials(float* x) {
  float m = -__builtin_inff();
#pragma unroll
  for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
  m = over_lanes<L>(m, [](float a, float b) { return fmaxf(a, b); });
  float z = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    x[v] = exp_below(x[v] - m);
    z += x[v];
  }
  return 1.0f / over_lanes<L>(z, Add{});
}

// Counts, sums and loss from all workgroups' (`groups` of them, in `p` and `n`), by one workgroup.
// lds_p, lds_n: kRouteThreads words each; they may be where p and n are.
__device__ inline void finish_route(const RouteArgs& a, const float* p, const int32_t* n,
                                    int groups, float* lds_p, int32_t* lds_n) {
  const int tid = threadIdx.x, E = a.E;
  // `split` threads for each expert
  int wide = 1;
  while (wide < E) wide *= 2;
  const int split = kRouteThreads / wide, e = tid % wide, s = tid / wide;
  float sum = 0.0f;
  int32_t count = 0;
  if (e < E) {
#pragma unroll 16
    for (int g = s; g < groups; g += split) {
      sum += p[(int64_t)g * E + e];
      count += n[(int64_t)g * (E + 1) + e];
    }
  }
  int32_t rows = 0;
  if (tid < 64) {
    for (int g = tid; g < groups; g += 64) rows += n[(int64_t)g * (E + 1) + E];
    rows = over_lanes<64>(rows, Add{});
  }
  __syncthreads();  // (p and n have been read)
  lds_p[tid] = sum;
  lds_n[tid] = count;
  __syncthreads();
  for (int d = split / 2; d > 0; d /= 2) {
    if (s < d) {
      lds_p[tid] += lds_p[tid + d * wide];
      lds_n[tid] += lds_n[tid + d * wide];
    }
    __syncthreads();
  }
  if (tid < E) a.counts[tid] = lds_n[tid];
  if (tid < 64) {
    int32_t all = 0;
    double l = 0.0;
    for (int i = tid; i < E; i += 64) {
      all += lds_n[i];
      l += (double)lds_n[i] * (double)lds_p[i];
    }
    all = over_lanes<64>(all, Add{});
    for (int d = 1; d < 64; d *= 2) l += __shfl_xor(l, d);
    if (tid == 0) {
      a.sums[0] = rows;
      a.sums[1] = all;
      *a.loss = all ? (float)(l * E / ((double)all * (double)rows)) : 0.0f;
    }
  }
}

template <class T, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void ex_route_kernel(RouteArgs a) {
  constexpr int COLS = L * V, WAVES = kRouteThreads / 64, PER = kRouteThreads / L;
  constexpr int WORDS = WAVES * COLS > kRouteThreads ? WAVES * COLS : kRouteThreads;
  __shared__ float lds_p[WORDS];
  __shared__ int32_t lds_n[kRouteThreads + 1];
  const int tid = threadIdx.x, lane = tid % L, wave = tid / 64;
  for (int i = tid; i <= a.E; i += kRouteThreads) lds_n[i] = 0;
  __syncthreads();
  float acc[V] = {};
  int32_t rows = 0;
  for (int64_t t = (int64_t)blockIdx.x * PER + tid / L; t < a.rows; t += (int64_t)gridDim.x * PER) {
    float x[V];
    load_logits<T, L, V>(a.X, t * a.ldx, a.E, lane, x);
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key_of(x[v]);
    uint32_t most = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) most = max(most, key[v]);
    most = over_lanes<L>(most, Most{});
    const bool on = (a.valid == nullptr || a.valid[t] != 0) && most > kKeyNoExpert;
    // (the probabilities are added before the search, which then has their registers)
    const float inv = exponentials<L, V>(x);
    if (on) {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += x[v] * inv;
      rows += lane == 0;
    }
    // the j-th best of the row is kept by its lane j
    const float top = of_key(most);
    uint32_t mine = 0;
    int expert = -1;
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) best = max(best, key[v]);
      best = over_lanes<L>(best, Most{});
      int at = COLS;
#pragma unroll
      for (int v = 0; v < V; ++v) at = min(at, key[v] == best ? column<L, V>(lane, v) : COLS);
      at = over_lanes<L>(at, Least{});
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (column<L, V>(lane, v) == at) key[v] = 0;
      if (lane == j && on && best > kKeyNoExpert) {
        mine = best;
        expert = at;
      }
    }
    // (a NaN is the largest, and makes the gates NaN as it does the probabilities)
    float gate = expert >= 0 ? exp_below(of_key(mine) - top) * inv : 0.0f;
    if (a.norm) {
      const float sum = over_lanes<L>(gate, Add{});
      if (expert >= 0) gate /= sum;
    }
    if (lane < a.k) {
      a.gates[t * a.k + lane] = gate;
      a.experts[t * a.k + lane] = expert;
    }
    if (expert >= 0) atomicAdd(&lds_n[expert], 1);
  }
  // the workgroup's sums: over the rows of a wave, then over the waves
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (L == 16) {
      acc[v] += __shfl_xor(acc[v], 16);
      acc[v] += __shfl_xor(acc[v], 32);
    }
    if ((tid & 63) < L) lds_p[wave * COLS + column<L, V>(lane, v)] = acc[v];
  }
  if (rows) atomicAdd(&lds_n[a.E], rows);
  __syncthreads();
  float sum = 0.0f;
  if (tid < a.E) {
    for (int w = 0; w < WAVES; ++w) sum += lds_p[w * COLS + tid];
  }
  if (gridDim.x > 1) {
    if (tid < a.E) a.part_p[(int64_t)blockIdx.x * a.E + tid] = sum;
    for (int i = tid; i <= a.E; i += kRouteThreads)
      a.part_n[(int64_t)blockIdx.x * (a.E + 1) + i] = lds_n[i];
    return;
  }
  __syncthreads();
  if (tid < a.E) lds_p[tid] = sum;
  __syncthreads();
  finish_route(a, lds_p, lds_n, 1, lds_p, lds_n);
}

__global__ __launch_bounds__(kRouteThreads) void ex_route_finish_kernel(RouteArgs a) {
  __shared__ float lds_p[kRouteThreads];
  __shared__ int32_t lds_n[kRouteThreads];
  finish_route(a, a.part_p, a.part_n, a.groups, lds_p, lds_n);
}

// dx_e = p_e (G_e - sum p G) with G_e = dloss E counts_e / (n sum counts), and of the chosen ones'
// gates: dgates_j more in G, or, where they were divided by their sum, gates_j (dgates_j - sum_i
// dgates_i gates_i) more in dx.
constexpr int kRouteGradThreads = 256;
template <class T, int L, int V>
__global__ __launch_bounds__(kRouteGradThreads) void ex_route_grad_kernel(RouteArgs a) {
  constexpr int PER = kRouteGradThreads / L;
  const int lane = threadIdx.x % L;
  const float n = (float)a.sums[0], all = (float)a.sums[1];
  const float unit = a.dloss != nullptr && all > 0 ? *a.dloss * ((float)a.E / n / all) : 0.0f;
  float coef[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = column<L, V>(lane, v);
    coef[v] = c < a.E ? unit * (float)a.counts[c] : 0.0f;
  }
  for (int64_t t = (int64_t)blockIdx.x * PER + threadIdx.x / L; t < a.rows;
       t += (int64_t)gridDim.x * PER) {
    float x[V], g[V];
    load_logits<T, L, V>(a.X, t * a.ldx, a.E, lane, x);
    int expert = -1;
    float add = 0.0f;
    if (lane < a.k && a.dgates != nullptr) {
      expert = a.experts[t * a.k + lane];
      if (expert >= 0) add = a.dgates[t * a.k + lane];
    }
    const float gate = expert >= 0 && a.norm ? a.gates[t * a.k + lane] : 0.0f;
    if (a.norm) add = gate * (add - over_lanes<L>(gate * add, Add{}));
    bool on = a.valid == nullptr || a.valid[t] != 0;
    uint32_t best = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) best = max(best, key_of(x[v]));
    on = on && over_lanes<L>(best, Most{}) > kKeyNoExpert;
    const float inv = exponentials<L, V>(x);
    float chosen[V] = {};
    for (int j = 0; j < a.k; ++j) {
      const int e = __shfl(expert, j, L);
      const float d = __shfl(add, j, L);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (column<L, V>(lane, v) == e) chosen[v] = d;
    }
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] *= inv;
      g[v] = a.norm ? coef[v] : coef[v] + chosen[v];
      dot += x[v] * g[v];
    }
    dot = over_lanes<L>(dot, Add{});
#pragma unroll
    for (int v = 0; v < V; ++v) {
      g[v] = on ? x[v] * (g[v] - dot) : 0.0f;
      if (on && a.norm) g[v] += chosen[v];
    }
    if constexpr (V == 1) {
      if (lane < a.E) ((typename T::type*)a.DX)[t * a.lddx + lane] = (typename T::type)g[0];
    } else {
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        const int c = column<L, V>(lane, q);
        store_row<4, T::CODE>(a.DX, t * a.lddx + c, a.E - c, T::CODE, g + q);
      }
    }
  }
}

}  // namespace gemmlp
