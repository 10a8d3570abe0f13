// Adapters of low rank, each for a group of rows: out = y + s_e (x A_e^T) B_e with A_e rank x K and
// B_e rank x N, and their gradients.  With u = s x A^T and v = s dout B^T,
//   out = y + u B,  dx = v A,  dA = v^T x,  dB = u^T dout,
// so that three kernels serve all of it: `down` (u, v: the contraction is the wide axis), `up`
// (out, dx: the contraction is the rank) and `grad` (dA, dB: it is the group's rows).  As A and B
// both have the wide axis contiguous, every kernel reads all of its operands in whole lines.
//
// u and v stay in FP32 between the kernels.  `down` multiplies 16-bit values by the 16-bit matrix
// instruction (exact products, FP32 sums).  In `up` and `grad` one operand is u or v: for bf16 it
// is cut into three bf16 parts of 8 bits each, whose sum it is exactly, and multiplied part by part
// by the 16-bit instruction; fp16, whose exponents end too early for such parts, and FP32 take the
// FP32 instruction.  Both operands of these kernels lie across the contraction: a lane loads 8 k of
// 8 neighbouring columns, which is all that its fragments need of either instruction, so that
// nothing moves between lanes, and neighbouring lanes load and store neighbouring columns.
#pragma once

#include "ex_common.h"

namespace gemmlp {

struct AdapterArgs {
  const void* X;         // down, grad: the rows
  const void* W;         // down, up: the adapters
  void* C;               // up, grad: the result
  const int32_t* offsets;
  const int64_t* order;
  const float* scale;
  const void* Y;
  float* U;              // [split][place][ldu], zeros past the rank
  float* part;           // grad: [split of rows][E][rank][N], where there are several
  int64_t ldx, ldw, stride_w, ldc, stride_c, ldy;
  int rows, N, K, E;
  int rank, ldu;
  int splits;            // of U
  int tiles_n;           // up, grad: blocks of columns
  int k_chunk;           // down: columns of a split
  int row_splits;        // grad
};

// The columns of U: whole fragments of 16, so that its loads need no bounds.
__host__ __device__ inline int u_columns(int rank) { return (rank + 15) / 16 * 16; }

__device__ __forceinline__ int64_t row_at(const AdapterArgs& a, int place) {
  const int64_t r = a.order[place];
  return min(max(r, (int64_t)0), (int64_t)a.rows - 1);
}

// Inclusive sums over the lanes of a wave, on the vector unit.
__device__ __forceinline__ int wave_scan(int v) {
  auto step = [&](auto ctrl, auto rows) {
    v += __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
  };
  using std::integral_constant;
  step(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr:1
  step(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});  // row_bcast:15
  step(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});  // row_bcast:31
  return v;
}

// The places of tile `id` of BM: adapter e's are offsets[e] .. offsets[e+1] - 1, and -1 has those
// before the first and from the last on.  Every wave looks for itself, 64 groups at a time (E of
// them and the two of none); false past the last tile.
struct Places {
  int e, first, end;
};
template <int BM>
__device__ inline bool find_places(const AdapterArgs& a, int id, Places& t) {
  const int lane = threadIdx.x & 63, groups = a.E + 2;
  for (int base = 0; base < groups; base += 64) {
    const int g = base + lane;
    int lo = 0, hi = 0;
    if (g < groups) {
      lo = g == 0 ? 0 : clamped_offset(a.offsets, g - 1, a.rows);
      hi = g == groups - 1 ? a.rows : clamped_offset(a.offsets, g, a.rows);
    }
    const int tiles = (max(hi - lo, 0) + BM - 1) / BM;
    const int upto = wave_scan(tiles);
    const uint64_t past = __ballot(upto > id);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int found = base + l;
      t.e = found == 0 || found == groups - 1 ? -1 : found - 1;
      t.first = __builtin_amdgcn_readlane(lo, l) +
                (id - __builtin_amdgcn_readlane(upto - tiles, l)) * BM;
      t.end = min(__builtin_amdgcn_readlane(hi, l), t.first + BM);
      return true;
    }
    id -= __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
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

// ------------------------------------------------------------------------------------ down
// u of 16 RW places and one split of K: RW waves have 16 places each, and 4 / RW share each wave's
// steps of K and add up through LDS.  The instruction's rows are the rank, its columns the places.
// RF: fragments of 16 of the rank.
//
// A step is 128 bytes of every row, loaded by eight neighbouring lanes, and turned into fragments by
// a tile of LDS of the wave's own, so that no barrier is needed: one wave's LDS instructions run in
// order.  (Fragments loaded as they are have their neighbouring lanes in 16 different rows, and the
// address unit takes 64 cycles for such a load instead of 16.)  The 16-byte groups of a row change
// places from row to row, which keeps both sides free of bank conflicts.  The loads of kDownDeep
// steps are always under way.
constexpr int kDownThreads = 256;
template <int RF>
constexpr int kDownDeep = RF == 1 ? 6 : RF == 2 ? 4 : RF == 4 ? 3 : 2;
__device__ __forceinline__ int group_at(int row, int c) {  // of 16 bytes, in the wave's tile
  return row * 8 + (c ^ ((row >> 1) & 7));
}
template <class T, int RF, int RW>
__global__ __launch_bounds__(kDownThreads) void ex_adapters_down_kernel(AdapterArgs a) {
  constexpr int PER = 16 / T::BYTES, STEP = kRowBytes / T::BYTES;
  constexpr int LD = RF * 16 + 4, KW = 4 / RW, DEEP = kDownDeep<RF>, ROWS = 2 * (1 + RF);
  __shared__ int4v tile[4][ROWS * 8 * 8];
  using Vec = Raw<T, PER>;
  Places t;
  const int split = blockIdx.x % a.splits;
  if (!find_places<16 * RW>(a, blockIdx.x / a.splits, t) || t.e < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const int place0 = t.first + 16 * (wave % RW), part = wave / RW;
  int4v* const mine = tile[wave];
  float4v acc[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) acc[f] = float4v{0, 0, 0, 0};
  if (place0 < t.end) {
    // the rows that this lane loads of: two of the places', then two of each fragment's
    const int r8 = lane >> 3, c8 = lane & 7;
    const typename T::type* from[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
      from[j] = (j < 2 ? (const typename T::type*)a.X +
                             row_at(a, min(place0 + 8 * j + r8, t.end - 1)) * a.ldx
                       : (const typename T::type*)a.W + t.e * a.stride_w +
                             min(8 * (j - 2) + r8, a.rank - 1) * a.ldw) + c8 * PER;
    const int first = (int)min((int64_t)split * a.k_chunk, (int64_t)a.K);
    const int end = first + min(a.k_chunk, a.K - first);
    Vec v[DEEP][ROWS];
    const int whole = (end - first) / STEP;  // steps of all waves; this one has every KW-th
    const int n = (whole - part + KW - 1) / KW;
    auto load = [&](int d, int i) {
      const int k = first + (part + i * KW) * STEP;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) v[d][j] = load_raw<T, PER>(from[j] + k);
    };
    auto multiply = [&](int d) {
#pragma unroll
      for (int j = 0; j < ROWS; ++j)
        mine[group_at(8 * j + r8, c8)] = __builtin_bit_cast(int4v, v[d][j]);
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Vec x = __builtin_bit_cast(Vec, mine[group_at(l16, g + 4 * h)]);
#pragma unroll
        for (int f = 0; f < RF; ++f) {
          const Vec w = __builtin_bit_cast(Vec, mine[group_at(16 * (f + 1) + l16, g + 4 * h)]);
          if constexpr (T::BYTES == 4) {
#pragma unroll
            for (int j = 0; j < PER; ++j) acc[f] = mma32(w[j], x[j], acc[f]);
          } else {
            acc[f] = mma16(w, x, acc[f]);
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    };
    int i = 0;
    if (n >= DEEP) {
#pragma unroll
      for (int d = 0; d < DEEP; ++d) load(d, d);
      for (; i + 2 * DEEP <= n; i += DEEP) {
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
          multiply(d);
          load(d, i + DEEP + d);
        }
      }
#pragma unroll
      for (int d = 0; d < DEEP; ++d) multiply(d);
      i += DEEP;
    }
#pragma unroll
    for (int d = 0; d < DEEP - 1; ++d)
      if (i + d < n) load(d, i + d);
#pragma unroll
    for (int d = 0; d < DEEP - 1; ++d)
      if (i + d < n) multiply(d);
    // the columns past the last whole step, by the wave whose turn it is
    const int rest = first + whole * STEP;
    if (rest < end && whole % KW == part) {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        v[0][j] = load_columns<T, PER, false>(from[j] - c8 * PER, rest + c8 * PER, end);
#pragma unroll
        for (int k = 0; k < PER; ++k)
          v[0][j][k] = rest + c8 * PER + k < end ? v[0][j][k] : (typename T::type)0.0f;
      }
      multiply(0);
    }
  }
  // (a wave's sums lie where its tile was)
  static_assert(16 * LD * 4 <= ROWS * 8 * kRowBytes, "the sums fit into the tile");
#pragma unroll
  for (int f = 0; f < RF; ++f) *(float4v*)((float*)mine + l16 * LD + 16 * f + 4 * g) = acc[f];
  __syncthreads();
  const float s = a.scale != nullptr ? a.scale[t.e] : 1.0f;
  float* u = a.U + (int64_t)split * a.rows * a.ldu;
  for (int i = tid; i < RW * 16 * RF * 4; i += kDownThreads) {
    const int row = i / (RF * 4), r = i % (RF * 4) * 4;
    float4v v = *(const float4v*)((const float*)tile[row / 16] + row % 16 * LD + r);
#pragma unroll
    for (int q = 1; q < KW; ++q)
      v += *(const float4v*)((const float*)tile[q * RW + row / 16] + row % 16 * LD + r);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = r + j < a.rank ? v[j] * s : 0.0f;
    if (t.first + row < t.end && r < a.ldu)
      *(float4v*)(u + (int64_t)(t.first + row) * a.ldu + r) = v;
  }
}

// ------------------------------------------------------------- contractions across both operands
// The instruction's columns are columns of the result, and 128 of these make eight fragments: column
// l of fragment j is 8 l + j.  A lane loads the eight columns of its l at once, and holds these eight
// of the result, of four rows.

// What a lane has of one operand in 32 k: 8 k (8 g + i) of 8 neighbouring columns.
template <class T>
struct Block8 {
  Raw<T, 8> v[8];  // v[i][j]: k = 8 g + i, column j; after turn(): v[j][i]
  __device__ __forceinline__ void turn() {
    if constexpr (T::BYTES == 2) {
      Block8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) o.v[j][i] = v[i][j];
      *this = o;
    }
  }
};

// The three bf16 parts of FP32 numbers, cut (not rounded) so that they add up exactly and no part
// passes bf16's range; Inf and NaN are in the first.
__device__ __forceinline__ void three_parts(const float (&u)[8], bf168v (&part)[3]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float rest = u[i];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const uint32_t top = __builtin_bit_cast(uint32_t, rest) & 0xffff0000u;
      part[p][i] = __builtin_bit_cast(__bf16, (uint16_t)(top >> 16));
      const float cut = __builtin_bit_cast(float, top);
      rest = rest == cut ? 0.0f : rest - cut;
    }
  }
}

// acc[j] += u x fragment j of `w` over 32 k, u the instruction's row l16.  bf16: w turned.
template <class T>
__device__ __forceinline__ void multiply_across(const Block8<T>& w, const float (&u)[8],
                                                float4v (&acc)[8]) {
  if constexpr (std::is_same_v<T, Bf16>) {
    bf168v part[3];
    three_parts(u, part);
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = mma16(part[p], w.v[j], acc[j]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = mma32(u[i], (float)w.v[i][j], acc[j]);
  }
}

// Four neighbours of U, the splits' sum: their loads are in flight together.
template <bool SPLIT>
__device__ __forceinline__ float4v u_at(const AdapterArgs& a, int64_t at) {
  const float* u = a.U + at;
  float4v v = *(const float4v*)u;
  if constexpr (!SPLIT) return v;
  const int64_t step = (int64_t)a.rows * a.ldu;
  for (int s = 1; s < a.splits; s += 4) {
    float4v w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = *(const float4v*)(u + min(s + q, a.splits - 1) * step);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (s + q < a.splits) v += w[q];
  }
  return v;
}

// -------------------------------------------------------------------------------------- up
// BM places x 512 columns, a wave 128 of them and 16 places at a time, B's part in registers (where
// that takes 128 of them or fewer).  NB: blocks of 32 of the rank.  BM is 16, or 64 where U has one
// split.
constexpr int kUpThreads = 256, kWaveCols = 128, kUpCols = 4 * kWaveCols;
template <class T, int NB, int BM, bool INSIDE>
__device__ __forceinline__ void up_columns(const AdapterArgs& a, const Places& t, int n0) {
  constexpr bool HOLD = NB * 32 * (T::BYTES / 2) <= 128 && BM > 16;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int c = n0 + 8 * l16;
  int64_t rows[BM / 16][4];  // of the results that this lane holds
#pragma unroll
  for (int i = 0; i < BM / 16; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      rows[i][q] = row_at(a, min(t.first + 16 * i + 4 * g + q, t.end - 1));
  const typename T::type* w = (const typename T::type*)a.W + max(t.e, 0) * a.stride_w;
  auto load_w = [&](int b, Block8<T>& o) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 32 * b + 8 * g + i;
      o.v[i] = load_columns<T, 8, INSIDE>(w + min(r, a.rank - 1) * a.ldw, c, a.N);
    }
  };
  auto finish_w = [&](int b, Block8<T>& o) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * b + 8 * g + i >= a.rank) o.v[i] = Raw<T, 8>{};
    if constexpr (std::is_same_v<T, Bf16>) o.turn();
  };
  auto load_u = [&](int b, int place, float4v (&u)[2]) {
    const int r = 32 * b + 8 * g;
    const int64_t at = (int64_t)place * a.ldu + (r < a.ldu ? r : 0);
    u[0] = u_at<BM == 16>(a, at), u[1] = u_at<BM == 16>(a, at + 4);
    if (r >= a.ldu) u[0] = u[1] = float4v{0, 0, 0, 0};
  };
  Raw<T, 8> y[2][4];
  auto load_y = [&](int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      y[i & 1][q] = load_columns<T, 8, INSIDE>((const typename T::type*)a.Y + rows[i][q] * a.ldy,
                                               c, a.N);
  };
  Block8<T> held[HOLD ? NB : 1];
  if (HOLD && t.e >= 0) {
#pragma unroll
    for (int b = 0; b < NB; ++b) load_w(b, held[b]);
  }
  if (a.Y != nullptr) load_y(0);
  if (HOLD && t.e >= 0) {
#pragma unroll
    for (int b = 0; b < NB; ++b) finish_w(b, held[b]);
  }
#pragma unroll
  for (int i = 0; i < BM / 16; ++i) {
    const int p0 = t.first + 16 * i;
    if (p0 >= t.end) break;
    float4v acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = float4v{0, 0, 0, 0};
    if (t.e >= 0) {
      float4v u[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) load_u(b, min(p0 + l16, t.end - 1), u[b]);
      // the next places' y is on its way while these are multiplied
      if (i + 1 < BM / 16 && a.Y != nullptr) load_y(i + 1 < BM / 16 ? i + 1 : i);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = u[b][k / 4][k % 4];
        if constexpr (HOLD) {
          multiply_across<T>(held[b], v, acc);
        } else {
          Block8<T> o;
          load_w(b, o);
          finish_w(b, o);
          multiply_across<T>(o, v, acc);
        }
      }
    } else if (i + 1 < BM / 16 && a.Y != nullptr) {
      load_y(i + 1 < BM / 16 ? i + 1 : i);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = a.Y != nullptr ? (float)y[i & 1][q][j] + acc[j][q] : acc[j][q];
      if (p0 + 4 * g + q < t.end)
        store_row<8, T::CODE>(a.C, rows[i][q] * a.ldc + c, INSIDE ? 8 : a.N - c, T::CODE, v);
    }
  }
}
template <class T, int NB, int BM>
__global__ __launch_bounds__(kUpThreads) void ex_adapters_up_kernel(AdapterArgs a) {
  Places t;
  if (!find_places<BM>(a, blockIdx.x / a.tiles_n, t)) return;
  const int n0 = __builtin_amdgcn_readfirstlane(blockIdx.x % a.tiles_n * kUpCols +
                                                (threadIdx.x >> 6) * kWaveCols);
  if (n0 + kWaveCols <= a.N) up_columns<T, NB, BM, true>(a, t, n0);
  else if (n0 < a.N) up_columns<T, NB, BM, false>(a, t, n0);
}

// ------------------------------------------------------------------------------------ grad
// 128 columns of RF * 16 rows of one adapter's gradient.  The waves take turns at 32 of the group's
// places and add up through LDS; row_splits workgroups share a group's places.
template <int RF>
struct GradShape {
  static constexpr int WAVES = RF <= 2 ? 8 : 4;
};
// What one wave adds of the places first + 32 wave, + 32 WAVES and so on.
template <class T, int RF, bool INSIDE>
__device__ __forceinline__ void grad_places(const AdapterArgs& a, int first, int end, int n0, int r0,
                                            float4v (&acc)[RF][8]) {
  constexpr int WAVES = GradShape<RF>::WAVES;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int64_t u_step = (int64_t)a.rows * a.ldu;
  for (int i0 = first + (threadIdx.x >> 6) * 32; i0 < end; i0 += WAVES * 32) {
    int64_t rows[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rows[i] = row_at(a, min(i0 + 8 * g + i, end - 1));
    Block8<T> o;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o.v[i] = load_columns<T, 8, INSIDE>((const typename T::type*)a.X + rows[i] * a.ldx,
                                          n0 + 8 * l16, a.N);
    float u[RF][8];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int i = 0; i < 8; ++i) u[f][i] = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
      float part[RF][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float* at = a.U + s * u_step + (int64_t)min(i0 + 8 * g + i, end - 1) * a.ldu + l16;
#pragma unroll
        for (int f = 0; f < RF; ++f) part[f][i] = at[min(r0 + 16 * f, a.ldu - 16)];
      }
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int i = 0; i < 8; ++i) u[f][i] += part[f][i];
    }
    if (i0 + 32 > end) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + 8 * g + i >= end) {
          o.v[i] = Raw<T, 8>{};
#pragma unroll
          for (int f = 0; f < RF; ++f) u[f][i] = 0.0f;
        }
    }
    if constexpr (std::is_same_v<T, Bf16>) o.turn();
#pragma unroll
    for (int f = 0; f < RF; ++f) multiply_across<T>(o, u[f], acc[f]);
  }
}
template <class T, int RF>
__global__ __launch_bounds__(GradShape<RF>::WAVES * 64) void ex_adapters_grad_kernel(AdapterArgs a) {
  constexpr int WAVES = GradShape<RF>::WAVES, N = RF * 8 * 4;
  __shared__ float red[WAVES / 2][N][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  // workgroups: columns, then row splits, then blocks of the rank, then adapters
  const int rb = (a.rank + RF * 16 - 1) / (RF * 16);
  int id = blockIdx.x;
  const int n0 = id % a.tiles_n * kWaveCols;
  id /= a.tiles_n;
  const int split = id % a.row_splits;
  id /= a.row_splits;
  const int r0 = id % rb * (RF * 16), e = id / rb;
  const int lo = clamped_offset(a.offsets, e, a.rows);
  const int len = max(clamped_offset(a.offsets, e + 1, a.rows) - lo, 0);
  const int first = lo + (int)((int64_t)len * split / a.row_splits);
  const int end = lo + (int)((int64_t)len * (split + 1) / a.row_splits);
  float4v acc[RF][8];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[f][j] = float4v{0, 0, 0, 0};
  if (n0 + kWaveCols <= a.N) grad_places<T, RF, true>(a, first, end, n0, r0, acc);
  else grad_places<T, RF, false>(a, first, end, n0, r0, acc);
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
  const int c = n0 + 8 * l16;
#pragma unroll
  for (int f = 0; f < RF; ++f) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = r0 + 16 * f + 4 * g + q;
      if (r >= a.rank) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[f][j][q];
      if (a.row_splits > 1) {
        const int64_t at = (((int64_t)split * a.E + e) * a.rank + r) * a.N + c;
        store_row<8, GEMM_LP_F32>(a.part, at, a.N - c, GEMM_LP_F32, v);
      } else {
        store_row<8, T::CODE>(a.C, e * a.stride_c + r * a.ldc + c, a.N - c, T::CODE, v);
      }
    }
  }
}

// The sum of the row splits' parts; a thread has eight columns.
template <class T>
__global__ __launch_bounds__(256) void ex_adapters_sum_kernel(AdapterArgs a) {
  const int per = (a.N + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.E * a.rank * per) return;
  const int64_t row = i / per;  // e * rank + r
  const int c = (int)(i - row * per) * 8, n = a.N - c;
  float v[8] = {};
  for (int s = 0; s < a.row_splits; ++s) {
    const float* part = a.part + ((int64_t)s * a.E * a.rank + row) * a.N;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += part[min(c + j, a.N - 1)];
  }
  const int e = (int)(row / a.rank), r = (int)(row - (int64_t)e * a.rank);
  store_row<8, T::CODE>(a.C, e * a.stride_c + r * a.ldc + c, n, T::CODE, v);
}

}  // namespace gemmlp
