// Adapters of low rank, each for a group of rows: out = y + s_e (x A_e^T) B_e with A_e rank x K and
// B_e rank x N, and their gradients.  With u = s x A^T and v = s dout B^T,
//   out = y + u B,  dx = v A,  dA = v^T x,  dB = u^T dout,
// so that three kernels serve all of it: `down` (u, v: the contraction is the wide axis), `up`
// (out, dx: the contraction is the rank) and `grad` (dA, dB: it is the group's rows).  As A and B
// both have the wide axis contiguous, every kernel reads all of its operands in whole lines.
//
// u and v stay in FP32 between the kernels.  `down` multiplies 16-bit values by the 16-bit matrix
// instruction (exact products, FP32 sums).  In `up` and `grad` one operand is u or v: for bf16 it
// is cut into three bf16 parts of 8 bits each, whose sum it is (but for what is below bf16's smallest
// step, 2^-133), and multiplied part by part by the 16-bit instruction; fp16, whose exponents end too early for such parts, and FP32 take the
// FP32 instruction.  Both operands of these kernels lie across the contraction: a lane loads 8 k of
// 8 neighbouring columns, which is all that its fragments need of either instruction, so that
// nothing moves between lanes, and neighbouring lanes load and store neighbouring columns.
//
// Bound by memory, and by how evenly the groups fill the chip (bf16, each pass on other rows):
//   down  8192 x 4096, rank 32: 22 us for 67 MB (3.0 TB/s) and 4 for the launch that joins the
//         splits, which make it the same for even and uneven groups; 4096 x 4096, rank 16: 10 us;
//         one token each for 24 adapters, rank 16: 5.1 us, the latency of three loads that wait for
//         each other
//   up    4096 x 11008, rank 16: 39 us for 180 MB (4.6 TB/s; a large copy reaches 5.0); 24 adapters
//         of one token beside 4096 columns: 6.3 us
//   grad  8192 x 4096, rank 32, both gradients in one launch: 43 us for 134 MB and 4.2 for the sums
//         (in two launches 26 and 4.3 each): 170 registers leave room for one workgroup a CU, which
//         lives 9 us, of which 3 are vector
//         instructions (u's parts, turning) and most of the rest the chain from the offsets to the
//         rows' numbers to the rows
// With one workgroup's loads guarded one by one (a branch each, at which all earlier ones have to
// arrive) `up` took 84 us where it takes 39.
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
  float* part;           // grad: [slot][rank][N], a slot for each run of the adapters with several
  int64_t ldx, ldw, stride_w, ldc, stride_c, ldy;
  int rows, N, K, E;
  int rank, ldu;
  int splits;            // of U
  int tiles_n;           // up, grad: blocks of columns
  int k_chunk;           // down: columns of a split
  int run, slots;        // grad: places of a run, and how many of them `part` has room for
};

// The columns of U: whole fragments of 16, so that its loads need no bounds.
__host__ __device__ inline int u_columns(int rank) { return (rank + 15) / 16 * 16; }

__device__ __forceinline__ int64_t row_at(const AdapterArgs& a, int place) {
  const int64_t r = a.order[place];
  return min(max(r, (int64_t)0), (int64_t)a.rows - 1);
}

// Tiles of bm in a group of len places.  (Unsigned, as a run of the gradient can be so long that the
// sum of the two passes 31 bits.)
__host__ __device__ constexpr int tiles_of(int len, int bm) {
  return (int)(((unsigned)len + (unsigned)bm - 1u) / (unsigned)bm);
}
static_assert(tiles_of(2147482623, 4194560) == 512 && tiles_of(2147482623, 2147482624) == 1 &&
                  tiles_of(0, 16) == 0 && tiles_of(16, 16) == 1 && tiles_of(17, 16) == 2,
              "also at the largest number of rows");

// The places of tile `id` of bm: adapter e's are offsets[e] .. offsets[e+1] - 1, and -1 has those
// before the first and from the last on.  Every wave looks for itself, 64 groups at a time; false
// past the last tile.  NONE: with the places of no adapter; otherwise of the adapters alone, one
// tile at least of each.
struct Places {
  int e, first, end;
  int tile, tiles;  // which of its adapter's, and how many that has
  int slot;         // (of the adapters alone) which of the tiles of those that have several
};
template <bool NONE>
__device__ inline bool find_places(const AdapterArgs& a, int bm, int id, Places& t) {
  const int lane = threadIdx.x & 63, groups = NONE ? a.E + 2 : a.E;
  int slots = 0;
  for (int base = 0; base < groups; base += 64) {
    // group g: from edge g to edge g + 1, of which the adapters have 0 .. E
    const int g = min(base + lane, groups - 1) - (NONE ? 1 : 0);
    int lo = clamped_offset(a.offsets, max(g, 0), a.rows);
    int hi = clamped_offset(a.offsets, min(g + 1, a.E), a.rows);
    if (NONE && g < 0) lo = 0;
    if (NONE && g >= a.E) hi = a.rows;
    hi = max(hi, lo);
    const int tiles = base + lane < groups ? max(tiles_of(hi - lo, bm), NONE ? 0 : 1) : 0;
    const int upto = wave_scan(tiles);
    const int several = !NONE && tiles > 1 ? tiles : 0, upto_slot = NONE ? 0 : wave_scan(several);
    const uint64_t past = __ballot(upto > id);
    if (past) {
      const int l = __builtin_ctzll(past);
      t.e = __builtin_amdgcn_readlane(g, l);
      if (NONE && t.e >= a.E) t.e = -1;
      t.tiles = __builtin_amdgcn_readlane(tiles, l);
      t.tile = id - (__builtin_amdgcn_readlane(upto, l) - t.tiles);
      if (!NONE)
        t.slot = slots + t.tile + __builtin_amdgcn_readlane(upto_slot, l) - __builtin_amdgcn_readlane(several, l);
      t.first = __builtin_amdgcn_readlane(lo, l) + t.tile * bm;
      t.end = t.first + min(__builtin_amdgcn_readlane(hi, l) - t.first, bm);
      return true;
    }
    id -= __builtin_amdgcn_readlane(upto, 63);
    if (!NONE) slots += __builtin_amdgcn_readlane(upto_slot, 63);
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

// The operands' wide axis has kLeastWide columns at least (the kernels of fewer are at the end), so
// that a load of as many can always be moved back into the row.
constexpr int kLeastWide = 8;

// ------------------------------------------------------------------------------------ down
// Columns c .. c + COUNT - 1 of a row that lie before `end`, at places that depend on c and `end`
// alone (which is all that a contraction needs), zeros at the others.
template <class T, int COUNT>
__device__ __forceinline__ Raw<T, COUNT> load_end(const typename T::type* row, int c, int end) {
  const int at = min(c, end - COUNT);
  Raw<T, COUNT> v = load_raw<T, COUNT>(row + at);
#pragma unroll
  for (int i = 0; i < COUNT; ++i) v[i] = at + i < c ? (typename T::type)0.0f : v[i];
  return v;
}

// u of 16 places and one split of K, whose steps four waves share; they add up through LDS.  The
// instruction's rows are the rank, its columns the places.  RF: fragments of 16 of the rank.
//
// A step is 128 bytes of every row, loaded by eight neighbouring lanes, and turned into fragments by
// a tile of LDS of the wave's own, so that no barrier is needed: one wave's LDS instructions run in
// order.  (Fragments loaded as they are have their neighbouring lanes in 16 different rows, and the
// address unit takes 64 cycles for such a load instead of 16.)  The 16-byte groups of a row change
// places from row to row, which keeps both sides free of bank conflicts.  The loads of kDownDeep
// steps are always under way.
constexpr int kDownThreads = 256;
template <int RF>
constexpr int kDownDeep = RF <= 2 ? 4 : RF == 4 ? 3 : 2;
__device__ __forceinline__ int group_at(int row, int c) {  // of 16 bytes, in the wave's tile
  return row * 8 + (c ^ ((row >> 1) & 7));
}
template <class T, int RF>
__global__ __launch_bounds__(kDownThreads) void ex_adapters_down_kernel(AdapterArgs a) {
  constexpr int PER = 16 / T::BYTES, STEP = kRowBytes / T::BYTES;
  constexpr int LD = RF * 16 + 4, KW = 4, DEEP = kDownDeep<RF>, ROWS = 2 * (1 + RF);
  __shared__ int4v tile[4][ROWS * 8 * 8];
  using Vec = Raw<T, PER>;
  Places t;
  const int split = blockIdx.x % a.splits;
  if (!find_places<true>(a, 16, blockIdx.x / a.splits, t) || t.e < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const int part = wave;
  int4v* const mine = tile[wave];
  float4v acc[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) acc[f] = float4v{0, 0, 0, 0};
  // the rows that this lane loads of: two of the places', then two of each fragment's
  const int r8 = lane >> 3, c8 = lane & 7;
  const typename T::type* from[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j)
    from[j] = (j < 2 ? (const typename T::type*)a.X +
                           row_at(a, min(t.first + 8 * j + r8, t.end - 1)) * a.ldx
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
  if (n > 0) {
    // (past the last step its loads are made once more: without a branch, at which all loads would
    // have to arrive, and without a second set of registers for what is left over)
#pragma unroll
    for (int d = 0; d < DEEP; ++d) load(d, min(d, n - 1));
    for (int i = 0; i < n; i += DEEP) {
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        if (i + d < n) multiply(d);
        load(d, min(i + d + DEEP, n - 1));
      }
    }
  }
  // the columns past the last whole step, by the wave whose turn it is
  const int rest = first + whole * STEP;
  if (rest < end && whole % KW == part) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
      v[0][j] = load_end<T, PER>(from[j] - c8 * PER, rest + c8 * PER, end);
    multiply(0);
  }
  // (a wave's sums lie where its tile was)
  static_assert(16 * LD * 4 <= ROWS * 8 * kRowBytes, "the sums fit into the tile");
#pragma unroll
  for (int f = 0; f < RF; ++f) *(float4v*)((float*)mine + l16 * LD + 16 * f + 4 * g) = acc[f];
  __syncthreads();
  const float s = a.scale != nullptr ? a.scale[t.e] : 1.0f;
  float* u = a.U + (int64_t)split * a.rows * a.ldu;
  for (int i = tid; i < 16 * RF * 4; i += kDownThreads) {
    const int row = i / (RF * 4), r = i % (RF * 4) * 4;
    float4v v = *(const float4v*)((const float*)tile[0] + row * LD + r);
#pragma unroll
    for (int q = 1; q < KW; ++q) v += *(const float4v*)((const float*)tile[q] + row * LD + r);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = r + j < a.rank ? v[j] * s : 0.0f;
    if (t.first + row < t.end && r < a.ldu)
      *(float4v*)(u + (int64_t)(t.first + row) * a.ldu + r) = v;
  }
}

// The same for 64 places, by eight waves: four of them, a group, have 16 places each and share the
// adapter's part of a step, of which each loads its share, in two slots of LDS in turn with one
// barrier a step; their own rows' part they turn by themselves.  The two groups share the steps of K.
// (With a copy for each wave the adapter's bytes, from the L2, take longer than the rows' from memory:
// rank 32 has two of them for each of the rows', and a CU gets 16 a cycle.)
constexpr int kWideThreads = 512, kWidePlaces = 64;
template <int RF>
constexpr int kWideDeep = RF <= 2 ? 4 : RF == 4 ? 3 : 2;
template <class T, int RF>
__global__ __launch_bounds__(kWideThreads, (RF <= 2 ? 4 : 2)) void ex_adapters_down_wide_kernel(
    AdapterArgs a) {
  constexpr int PER = 16 / T::BYTES, STEP = kRowBytes / T::BYTES, DEEP = kWideDeep<RF>;
  constexpr int RW = kWidePlaces / 16, KG = 8 / RW, WROWS = RF * 16, LD = RF * 16 + 4;
  constexpr int OWN = (WROWS / 8 + RW - 1) / RW;  // loads of eight adapter rows a wave makes
  __shared__ int4v rows_tile[8][16 * 8];
  __shared__ int4v rank_tile[KG][2][WROWS * 8];
  using Vec = Raw<T, PER>;
  Places t;
  const int split = blockIdx.x % a.splits;
  if (!find_places<true>(a, kWidePlaces, blockIdx.x / a.splits, t) || t.e < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const int rw = wave % RW, kg = wave / RW;
  const int r8 = lane >> 3, c8 = lane & 7, place0 = t.first + 16 * rw;
  int4v* const mine = rows_tile[wave];
  float4v acc[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) acc[f] = float4v{0, 0, 0, 0};
  const typename T::type* from[2 + OWN];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    from[j] = (const typename T::type*)a.X +
              row_at(a, min(place0 + 8 * j + r8, t.end - 1)) * a.ldx + c8 * PER;
#pragma unroll
  for (int j = 0; j < OWN; ++j)
    from[2 + j] = (const typename T::type*)a.W + t.e * a.stride_w +
                  min(8 * (rw + RW * j) + r8, a.rank - 1) * a.ldw + c8 * PER;
  const bool owns = 8 * rw < WROWS;  // (16 ranks are two waves' loads)
  const int first = (int)min((int64_t)split * a.k_chunk, (int64_t)a.K);
  const int end = first + min(a.k_chunk, a.K - first);
  const int n = (end - first) / (STEP * KG);  // whole steps of every group
  Vec v[DEEP][2 + OWN];
  auto load = [&](int d, int i) {
#pragma unroll
    for (int j = 0; j < 2 + OWN; ++j)
      v[d][j] = load_raw<T, PER>(from[j] + first + (i * KG + kg) * STEP);
  };
  auto multiply = [&](int d, int i) {
    int4v* const shared = rank_tile[kg][i & 1];
#pragma unroll
    for (int j = 0; j < 2; ++j) mine[group_at(8 * j + r8, c8)] = __builtin_bit_cast(int4v, v[d][j]);
    if (owns) {
#pragma unroll
      for (int j = 0; j < OWN; ++j)
        shared[group_at(8 * (rw + RW * j) + r8, c8)] = __builtin_bit_cast(int4v, v[d][2 + j]);
    }
    // LDS alone: the loads of later steps stay under way
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const Vec x = __builtin_bit_cast(Vec, mine[group_at(l16, g + 4 * h)]);
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        const Vec w = __builtin_bit_cast(Vec, shared[group_at(16 * f + l16, g + 4 * h)]);
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
  if (n > 0) {
    // (as above)
#pragma unroll
    for (int d = 0; d < DEEP; ++d) load(d, min(d, n - 1));
    for (int i = 0; i < n; i += DEEP) {
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        if (i + d < n) multiply(d, i + d);
        load(d, min(i + d + DEEP, n - 1));
      }
    }
  }
  if (first + n * KG * STEP < end) {  // the columns past the last whole step of all groups
    const int k0 = first + (n * KG + kg) * STEP + c8 * PER;
#pragma unroll
    for (int j = 0; j < 2 + OWN; ++j) v[0][j] = load_end<T, PER>(from[j] - c8 * PER, k0, end);
    multiply(0, n);
  }
  // the groups' sums meet where the adapter's slots were
  static_assert((KG - 1) * RW * 16 * LD * 4 <= (int)sizeof(rank_tile), "they fit");
  __syncthreads();
  float* const sums = (float*)rank_tile;  // [group - 1][place][LD]
  if (kg > 0) {
#pragma unroll
    for (int f = 0; f < RF; ++f)
      *(float4v*)(sums + ((kg - 1) * RW * 16 + rw * 16 + l16) * LD + 16 * f + 4 * g) = acc[f];
  }
  __syncthreads();
  if (kg > 0) return;
  const float s = a.scale != nullptr ? a.scale[t.e] : 1.0f;
  float* u = a.U + (int64_t)split * a.rows * a.ldu + (int64_t)(place0 + l16) * a.ldu;
#pragma unroll
  for (int f = 0; f < RF; ++f) {
    const int r = 16 * f + 4 * g;
#pragma unroll
    for (int q = 1; q < KG; ++q)
      acc[f] += *(const float4v*)(sums + ((q - 1) * RW * 16 + rw * 16 + l16) * LD + r);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[f][j] = r + j < a.rank ? acc[f][j] * s : 0.0f;
    if (place0 + l16 < t.end && r < a.ldu) *(float4v*)(u + r) = acc[f];
  }
}

// The splits' sum, in the first one's place; a thread has four numbers.
__global__ __launch_bounds__(256) void ex_adapters_join_kernel(AdapterArgs a) {
  const int64_t n = (int64_t)a.rows * a.ldu, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  float4v v = *(const float4v*)(a.U + i);
#pragma unroll 8
  for (int s = 1; s < a.splits; ++s) v += *(const float4v*)(a.U + s * n + i);
  *(float4v*)(a.U + i) = v;
}

// ------------------------------------------------------------- contractions across both operands
// The instruction's columns are columns of the result, and 128 of these make eight fragments: column
// l of fragment j is 8 l + j.  A lane loads the eight columns of its l at once, and holds these eight
// of the result, of four rows.

// What a lane has of one operand in 32 k: 8 k (8 g + i) of CF neighbouring columns.
template <class T, int CF = 8>
struct Block8 {
  Raw<T, CF> v[8];  // v[i][j]: k = 8 g + i, column j; after turn(): v[j][i]
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

// The three bf16 parts of FP32 numbers, cut (not rounded) so that no part passes bf16's range.  They
// add up exactly from 2^-110 on; below, what the last has no steps for is lost, less than 2^-133.  Inf and NaN are in the first.  (A part may be 0, and 0 times Inf is NaN: an Inf
// of the other operand does not come out as one.)
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
template <class T, int CF>
__device__ __forceinline__ void multiply_across(const Block8<T, CF>& w, const float (&u)[8],
                                                float4v (&acc)[CF]) {
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
      for (int j = 0; j < CF; ++j) acc[j] = mma32(u[i], (float)w.v[i][j], acc[j]);
  }
}

// -------------------------------------------------------------------------------------- up
// A wave has 128 columns, and 16 places at a time: it reads their u and their rows of y, and B's part
// is there already.  Up to rank 32 that part is in the wave's registers, a workgroup is a wave, and
// it goes through BM places; past it four waves have 16 places each, and share B's part in LDS.
constexpr int kWaveCols = 128;

template <class T>
struct UpColumns {
  const AdapterArgs& a;
  const Places& t;
  int l16, g, c;

  __device__ __forceinline__ UpColumns(const AdapterArgs& args, const Places& places, int n0)
      : a(args), t(places), l16(threadIdx.x & 15), g(threadIdx.x >> 4 & 3),
        // (columns past the last are computed once more as the last ones)
        c(min(n0 + 8 * (int)(threadIdx.x & 15), args.N - 8)) {}

  // Ranks 32 b .. of the columns, zeros past the last.
  __device__ __forceinline__ void load(int b, Block8<T>& o) const {
    const typename T::type* w = (const typename T::type*)a.W + max(t.e, 0) * a.stride_w + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = load_raw<T, 8>(w + min(32 * b + 8 * g + i, a.rank - 1) * a.ldw);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * b + 8 * g + i >= a.rank) o.v[i] = Raw<T, 8>{};
    if constexpr (std::is_same_v<T, Bf16>) o.turn();
  }
  // Eight of u for place l16 of those from p0 on; zeros past the rank.
  __device__ __forceinline__ void load_u(int p0, int b, float (&v)[8]) const {
    const int r = 32 * b + 8 * g;
    const float* at = a.U + (int64_t)min(p0 + l16, t.end - 1) * a.ldu + (r < a.ldu ? r : 0);
    const int64_t step = (int64_t)a.rows * a.ldu;
    float4v u[2] = {*(const float4v*)at, *(const float4v*)(at + 4)};
    for (int s = 1; s < a.splits; s += 4) {  // (their loads together, four splits at a time)
      float4v more[4][2];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          more[k][h] = *(const float4v*)(at + min(s + k, a.splits - 1) * step + 4 * h);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (s + k < a.splits) u[0] += more[k][0], u[1] += more[k][1];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = r < a.ldu ? u[k / 4][k % 4] : 0.0f;
  }
  // 16 places from p0 on; row_of: the number of row lane + first; sum(acc) adds u B.
  template <class F>
  __device__ __forceinline__ void places(int p0, int first, int row_of, F sum) const {
    int64_t row[4];  // of the results that this lane holds
    Raw<T, 8> y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) row[q] = __shfl(row_of, min(p0 + 4 * g + q, t.end - 1) - first);
    if (a.Y != nullptr) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        y[q] = load_raw<T, 8>((const typename T::type*)a.Y + row[q] * a.ldy + c);
    }
    // (y + -0 is y, its sign too where it is 0)
    const float none = a.Y != nullptr && t.e < 0 ? -0.0f : 0.0f;
    float4v acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = float4v{none, none, none, none};
    if (t.e >= 0) sum(acc);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = a.Y != nullptr ? (float)y[q][j] + acc[j][q] : acc[j][q];
      if (p0 + 4 * g + q < t.end)
        store_row<8, T::CODE>(a.C, row[q] * a.ldc + c, 8, T::CODE, v);
    }
  }
};

// Rank 32 or less.  BM: 16, 32 or 64.
template <class T, int BM>
__global__ __launch_bounds__(64, (std::is_same_v<T, Bf16> ? 4 : T::BYTES == 2 ? 3 : 2)) void
ex_adapters_up_kernel(AdapterArgs a) {
  Places t;
  if (!find_places<true>(a, BM, blockIdx.x / a.tiles_n, t)) return;
  const UpColumns<T> w(a, t, blockIdx.x % a.tiles_n * kWaveCols);
  const int row_of = (int)row_at(a, min(t.first + ((int)threadIdx.x & (BM - 1)), t.end - 1));
  Block8<T> held;
  if (t.e >= 0) w.load(0, held);
  for (int p0 = t.first; p0 < t.end; p0 += 16)
    w.places(p0, t.first, row_of, [&](float4v (&acc)[8]) {
      float u[8];
      w.load_u(p0, 0, u);
      multiply_across<T>(held, u, acc);
    });
}

// Rank 128 or less: 64 places a workgroup.
template <class T>
__global__ __launch_bounds__(256) void ex_adapters_up_deep_kernel(AdapterArgs a) {
  __shared__ Raw<T, 8> shared[4][8][64];
  Places t;
  if (!find_places<true>(a, 64, blockIdx.x / a.tiles_n, t)) return;
  const UpColumns<T> w(a, t, blockIdx.x % a.tiles_n * kWaveCols);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row_of = (int)row_at(a, min(t.first + lane, t.end - 1));
  if (t.e >= 0 && 32 * wave < a.rank) {
    Block8<T> o;
    w.load(wave, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) shared[wave][i][lane] = o.v[i];
  }
  __syncthreads();
  const int p0 = t.first + 16 * wave;
  if (p0 >= t.end) return;
  w.places(p0, t.first, row_of, [&](float4v (&acc)[8]) {
    for (int b = 0; 32 * b < a.rank; ++b) {
      float u[8];
      w.load_u(p0, b, u);
      Block8<T> o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = shared[b][i][lane];
      multiply_across<T>(o, u, acc);
    }
  });
}

// ------------------------------------------------------------------------------------ grad
// One gradient, or both of a step in one launch: the first `wgs` workgroups have the first.
struct GradArgs {
  AdapterArgs set[2];
  int wgs;
};

// Columns of a workgroup: 64 past rank 32, as with 128 the sums take all registers of a SIMD's only
// wave.  (8192 x 4096, bf16, rank 64, four and 64 even adapters, when it was chosen: 57 and 124 us, 64 and
// 171 with 128; FP32, 4096 x 4096 of eight, 55 and 71.  Up to rank 32 128 need fewer instructions: bf16, rank 16, 37 us, 40
// with 64.)
__host__ __device__ constexpr int grad_columns(int rank) { return rank <= 32 ? 128 : 64; }

// These columns of RF * 16 rows of one adapter's gradient, from a run of its places.  The waves take
// turns at 32 of these and add up through LDS.  An adapter with one run has its result; those of one
// with several are added by another launch.  (Runs of one length, however the places are shared out:
// with as many for each adapter the largest one decides.)
template <int RF, int WAVES>
struct GradShape {
  static constexpr int CF = grad_columns(RF * 16) / 16;  // fragments of the columns
  static constexpr int LD = RF * 16 + 4;                 // numbers of a place in LDS
  static constexpr int N = RF * CF * 4;                  // numbers of a lane's sums
  static constexpr int U = WAVES * 32 * LD, SUMS = WAVES / 2 * N * 64;
};
// What one wave adds of the places first + 32 wave, + 32 WAVES and so on.  u and the rows' numbers
// come by whole lines, through LDS of the wave's own (lds: 32 LD numbers).
template <class T, int RF, int WAVES>
__device__ __forceinline__ void grad_places(const AdapterArgs& a, int first, int end, int c, int r0,
                                            float* lds,
                                            float4v (&acc)[RF][GradShape<RF, WAVES>::CF]) {
  constexpr int LD = GradShape<RF, WAVES>::LD, CF = GradShape<RF, WAVES>::CF;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int64_t u_step = (int64_t)a.rows * a.ldu;
  for (int i0 = first + (threadIdx.x >> 6) * 32; i0 < end; i0 += WAVES * 32) {
    const int row_of = (int)row_at(a, min(i0 + (lane & 31), end - 1));
    // u: 4 RF lanes load a place's 16 RF numbers
    constexpr int LANES = 4 * RF, PLACES = 64 / LANES;
    float4v part[32 / PLACES];
    const int ur = min(r0 + lane % LANES * 4, a.ldu - 4);
    auto load_u = [&](int s, float4v (&to)[32 / PLACES]) {
#pragma unroll
      for (int j = 0; j < 32 / PLACES; ++j)
        to[j] = *(const float4v*)(a.U + s * u_step +
                                  (int64_t)min(i0 + j * PLACES + lane / LANES, end - 1) * a.ldu + ur);
    };
    load_u(0, part);
    Block8<T, CF> o;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o.v[i] = load_raw<T, CF>((const typename T::type*)a.X +
                              (int64_t)__shfl(row_of, 8 * g + i) * a.ldx + c);
    for (int s = 1; s < a.splits; ++s) {
      float4v more[32 / PLACES];
      load_u(s, more);
#pragma unroll
      for (int j = 0; j < 32 / PLACES; ++j) part[j] += more[j];
    }
#pragma unroll
    for (int j = 0; j < 32 / PLACES; ++j) {
      const int place = j * PLACES + lane / LANES;
      // (the places past the last, and the numbers past u's columns, add nothing)
      if (i0 + place >= end || r0 + lane % LANES * 4 >= a.ldu) part[j] = float4v{0, 0, 0, 0};
      *(float4v*)(lds + place * LD + lane % LANES * 4) = part[j];
    }
    if (i0 + 32 > end) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + 8 * g + i >= end) o.v[i] = Raw<T, CF>{};
    }
    __builtin_amdgcn_wave_barrier();
    if constexpr (std::is_same_v<T, Bf16> && RF == 4) {
      bf168v w[CF];  // (the columns held, one fragment of u cut at a time)
#pragma unroll
      for (int j = 0; j < CF; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[j][i] = o.v[i][j];
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        float u[8];
        bf168v parts[3];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = lds[(8 * g + i) * LD + 16 * f + l16];
        three_parts(u, parts);
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int j = 0; j < CF; ++j) acc[f][j] = mma16(parts[p], w[j], acc[f][j]);
      }
    } else if constexpr (std::is_same_v<T, Bf16>) {
      bf168v parts[RF][3];
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = lds[(8 * g + i) * LD + 16 * f + l16];
        three_parts(u, parts[f]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // (one fragment turned at a time: 32 registers fewer)
        bf168v w;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = o.v[i][j];
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int f = 0; f < RF; ++f) acc[f][j] = mma16(parts[f][p], w, acc[f][j]);
      }
    } else {
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = lds[(8 * g + i) * LD + 16 * f + l16];
        multiply_across<T>(o, u, acc[f]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}
template <class T, int RF, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void ex_adapters_grad_kernel(
    GradArgs args) {
  const bool second = (int)blockIdx.x >= args.wgs;
  const AdapterArgs& a = args.set[second ? 1 : 0];
  using Shape = GradShape<RF, WAVES>;
  constexpr int N = Shape::N, LD = Shape::LD, CF = Shape::CF;
  // (the waves' u, and then their sums)
  __shared__ alignas(16) float shared[Shape::U > Shape::SUMS ? Shape::U : Shape::SUMS];
  float (*const red)[N][64] = (float (*)[N][64])shared;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  // workgroups: columns, then blocks of the rank, then runs
  const int rb = (a.rank + RF * 16 - 1) / (RF * 16);
  int id = (int)blockIdx.x - (second ? args.wgs : 0);
  const int n0 = id % a.tiles_n * (16 * CF);
  id /= a.tiles_n;
  const int r0 = id % rb * (RF * 16);
  id /= rb;
  Places t;
  if (!find_places<false>(a, a.run, id, t)) return;
  const int first = t.first, end = t.end;
  float4v acc[RF][CF];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int j = 0; j < CF; ++j) acc[f][j] = float4v{0, 0, 0, 0};
  float* const lds = shared + wave * 32 * LD;
  // (columns past the last are computed once more as the last ones)
  const int c = min(n0 + CF * l16, a.N - CF);
  grad_places<T, RF, WAVES>(a, first, end, c, r0, lds, acc);
  __syncthreads();
  for (int d = WAVES / 2; d > 0; d /= 2) {
    if (wave >= d && wave < 2 * d) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave - d][i][lane] = acc[i / (4 * CF)][i / 4 % CF][i % 4];
    }
    __syncthreads();
    if (wave < d) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i / (4 * CF)][i / 4 % CF][i % 4] += red[wave][i][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int f = 0; f < RF; ++f) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = r0 + 16 * f + 4 * g + q;
      if (r >= a.rank) continue;
      float v[CF];
#pragma unroll
      for (int j = 0; j < CF; ++j) v[j] = acc[f][j][q];
      if (t.tiles > 1) {
        // (offsets that overlap would give more slots than there are)
        const int64_t slot = min(t.slot, a.slots - 1);
        store_row<CF, GEMM_LP_F32>(a.part, (slot * a.rank + r) * a.N + c, CF, GEMM_LP_F32, v);
      } else {
        store_row<CF, T::CODE>(a.C, t.e * a.stride_c + r * a.ldc + c, CF, T::CODE, v);
      }
    }
  }
}

// The sums of the adapters that have several runs.  A workgroup has 2048 neighbouring values of one
// adapter's gradient, a thread eight of one row.
template <class T>
__global__ __launch_bounds__(256) void ex_adapters_sum_kernel(GradArgs args) {
  const bool second = (int)blockIdx.x >= args.wgs;
  const AdapterArgs& a = args.set[second ? 1 : 0];
  const unsigned wg = blockIdx.x - (second ? args.wgs : 0);
  const int per = (a.N + 7) / 8;
  const int64_t blocks = ((int64_t)a.rank * per + 255) / 256;
  const int e = (int)(wg / blocks);
  const int64_t i = (wg - e * blocks) * 256 + threadIdx.x;
  // its first slot: the runs of the adapters before it that have several
  int before = 0, runs = 0;
  for (int base = 0; base <= e; base += 64) {
    const int g = base + (threadIdx.x & 63);
    const int lo = clamped_offset(a.offsets, min(g, e), a.rows);
    const int len = max(clamped_offset(a.offsets, min(g, e) + 1, a.rows) - lo, 0);
    const int n = max(tiles_of(len, a.run), 1);
    // (offsets that overlap would count more slots than there are)
    before = min(before + __builtin_amdgcn_readlane(wave_scan(g < e && n > 1 ? n : 0), 63), a.slots);
    runs = __builtin_amdgcn_readfirstlane(__shfl(n, e - base));  // (of the last turn)
  }
  if (runs == 1 || i >= (int64_t)a.rank * per) return;
  const int r = (int)(i / per), c = min((int)(i - (int64_t)r * per) * 8, a.N - 8);
  float v[8] = {};
#pragma unroll 4
  for (int s = 0; s < runs; ++s) {
    const int at = min(before + s, a.slots - 1);
    const float* part = a.part + ((int64_t)at * a.rank + r) * a.N;
    const Raw<F32, 8> w = load_raw<F32, 8>(part + c);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += w[j];
  }
  store_row<8, T::CODE>(a.C, e * a.stride_c + r * a.ldc + c, 8, T::CODE, v);
}

// ----------------------------------------------------------------- fewer than kLeastWide columns
// u, 16 places and one split, a thread a number.  (The other splits are zeros.)
template <class T>
__global__ __launch_bounds__(256) void ex_adapters_down_few_kernel(AdapterArgs a) {
  Places t;
  const int split = blockIdx.x % a.splits;
  if (!find_places<true>(a, 16, blockIdx.x / a.splits, t) || t.e < 0) return;
  for (int i = threadIdx.x; i < (t.end - t.first) * a.ldu; i += 256) {
    const int place = t.first + i / a.ldu, r = i % a.ldu;
    float v = 0.0f;
    if (r < a.rank && split == 0) {
      const typename T::type* x = (const typename T::type*)a.X + row_at(a, place) * a.ldx;
      const typename T::type* w = (const typename T::type*)a.W + t.e * a.stride_w + r * a.ldw;
      for (int k = 0; k < a.K; ++k) v = fmaf((float)x[k], (float)w[k], v);
      if (a.scale != nullptr) v *= a.scale[t.e];
    }
    a.U[((int64_t)split * a.rows + place) * a.ldu + r] = v;
  }
}
// The result, 16 places, a thread a number.
template <class T>
__global__ __launch_bounds__(256) void ex_adapters_up_few_kernel(AdapterArgs a) {
  Places t;
  if (!find_places<true>(a, 16, blockIdx.x, t)) return;
  for (int i = threadIdx.x; i < (t.end - t.first) * a.N; i += 256) {
    const int place = t.first + i / a.N, n = i % a.N;
    const int64_t row = row_at(a, place);
    float v = a.Y != nullptr && t.e < 0 ? -0.0f : 0.0f;  // (as above)
    if (t.e >= 0) {
      for (int r = 0; r < a.rank; ++r) {
        float u = 0.0f;
        for (int s = 0; s < a.splits; ++s) u += a.U[((int64_t)s * a.rows + place) * a.ldu + r];
        v = fmaf(u, (float)((const typename T::type*)a.W)[t.e * a.stride_w + r * a.ldw + n], v);
      }
    }
    if (a.Y != nullptr) v += (float)((const typename T::type*)a.Y)[row * a.ldy + n];
    ((typename T::type*)a.C)[row * a.ldc + n] = (typename T::type)v;
  }
}
// One row of one adapter's gradient, its places shared by the threads.
template <class T>
__global__ __launch_bounds__(256) void ex_adapters_grad_few_kernel(AdapterArgs a) {
  __shared__ float part[4][kLeastWide];
  const int e = blockIdx.x / a.rank, r = blockIdx.x % a.rank, tid = threadIdx.x;
  const int lo = clamped_offset(a.offsets, e, a.rows), hi = clamped_offset(a.offsets, e + 1, a.rows);
  float v[kLeastWide] = {};
  for (int place = lo + tid; place < hi; place += 256) {
    const typename T::type* x = (const typename T::type*)a.X + row_at(a, place) * a.ldx;
    float u = 0.0f;
    for (int s = 0; s < a.splits; ++s) u += a.U[((int64_t)s * a.rows + place) * a.ldu + r];
#pragma unroll
    for (int n = 0; n < kLeastWide; ++n)
      if (n < a.N) v[n] = fmaf(u, (float)x[n], v[n]);
  }
#pragma unroll
  for (int n = 0; n < kLeastWide; ++n) {
    v[n] = over_lanes<64>(v[n], Add{});
    if ((tid & 63) == 0) part[tid >> 6][n] = v[n];
  }
  __syncthreads();
  if (tid < a.N)
    ((typename T::type*)a.C)[e * a.stride_c + r * a.ldc + tid] =
        (typename T::type)((part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]));
}

}  // namespace gemmlp
