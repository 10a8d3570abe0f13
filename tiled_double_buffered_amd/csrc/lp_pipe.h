// The product kernel: tiles of operands whose rows start at multiples of 4 bytes go from
// memory straight into LDS (gfx950's direct-to-LDS loads), two slots in turn, one barrier a
// K step.  (Three or four slots, with fewer workgroups on a CU, were 1.1 to 1.4 times slower.)
// Tiles of other operands pass through registers (STAGED) on the way.
//
// A K step is 128 bytes of every row where k is contiguous (128 8-bit, 64 16-bit, 32 32-bit
// values), so that all types share one LDS layout:
//   k contiguous: rows of 128 bytes whose 16-byte groups change places from row to row;
//   rows contiguous (the operand's k is the slow axis), 16-bit: k rows of R values, read
//     through the transposing LDS load, which hands each lane four k of one column; the 32
//     bytes of 16 columns at position j lie at j ^ f(k), so that the eight k rows that half a
//     wave reads (k mod 4 and k / 8 mod 2 vary) fall into different banks;
//   rows contiguous, 32-bit: k rows of R values as they are; a lane reads four (two)
//     neighbouring columns of one k, which are as many 16-column fragments, column 4 i + q the
//     i-th of the q-th, and the epilogue undoes that order.
// The copies write LDS in lane order, so each lane fetches what belongs at its place.
//
// Accumulators are transposed (D's rows are columns of C): a lane holds four neighbouring
// columns of one row of C and stores them at once.
//
// What bounds it: with many tiles the copies (16 cycles of the CU's address unit for each KiB;
// 128 x 128 tiles need as many cycles for them as for their products in 16 bits, 1090 TFLOP/s in
// bf16 at 8192^3), with few rows the reading of B (16 rows of 14 of 64 experts, 4096 x 2048 in
// bf16: 58 us, 4.05 TB/s; torch.sum reads as much memory at 3.5), with little work the latency of
// a step, which four wave groups on one tile share (1 x 11008 x 4096 in 8 bits: 15 us, 21 with one
// group).  8-bit values: 1.16 PFLOP/s at 8192 x 4096 x 4096 (237 us; with a scale for each column
// 263, with exponents 258), bound by the conversions beside the products, the matrix cores busy
// 56 %.  FP32: 139 TFLOP/s of 157 on 128 x 128 tiles, 132 on 64 x 64.
#pragma once

#include <type_traits>

#include "lp_common.h"

namespace gemmlp {

typedef __attribute__((address_space(3))) char lds_char;
typedef short short4v __attribute__((ext_vector_type(4)));

constexpr uint32_t kMaxRange = 0xFFFFFFF0u;
constexpr int kBufferWord3 = 0x00020000;  // untyped 32-bit data

__device__ __forceinline__ int4v buffer_words(const char* base, int64_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  int4v r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
  // rounded up to whole words: the range check goes by the word, and the last one, aligned,
  // holds a byte of the operand
  const int64_t n = bytes <= 0 ? 0 : (bytes + 3) & ~(int64_t)3;
  r[2] = __builtin_amdgcn_readfirstlane((int)(uint32_t)min(n, (int64_t)kMaxRange));
  r[3] = kBufferWord3;
  // a load may read a scalar that vector code wrote five wait states later, and the compiler
  // does not see the loads below
  asm volatile("s_nop 4" : "+s"(r));
  return r;
}

// The descriptors of an operand's K steps, one after another, by scalar arithmetic alone (a wave
// that computes them between its products holds the matrix cores up).
struct Walk {
  uint32_t lo, hi;   // base of the next step
  uint32_t rem_lo;   // bytes from there on, rounded up to whole words
  int rem_hi;
  uint32_t step_lo, step_hi;
  static __device__ __forceinline__ uint32_t scalar(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)x);
  }
  __device__ __forceinline__ void init(const char* base, int64_t left, int64_t step) {
    const uint64_t b = (uint64_t)(uintptr_t)base, n = (uint64_t)((left + 3) & ~(int64_t)3);
    lo = scalar((uint32_t)b), hi = scalar((uint32_t)(b >> 32));
    rem_lo = scalar((uint32_t)n), rem_hi = (int)scalar((uint32_t)(n >> 32));
    step_lo = scalar((uint32_t)step), step_hi = scalar((uint32_t)((uint64_t)step >> 32));
    // a load may read a scalar that vector code wrote five wait states later, and the compiler
    // does not see the loads
    asm volatile("s_nop 4" : "+s"(lo), "+s"(hi), "+s"(rem_lo), "+s"(rem_hi));
  }
  __device__ __forceinline__ int4v next() {
    int4v r;
    r[0] = (int)lo;
    r[1] = (int)hi;
    uint32_t n = rem_lo;
    n = rem_hi > 0 ? kMaxRange : n;
    n = rem_hi < 0 ? 0u : n;
    r[2] = (int)n;
    r[3] = kBufferWord3;
    const uint64_t b = ((uint64_t)hi << 32 | lo) + ((uint64_t)step_hi << 32 | step_lo);
    lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
    const uint64_t m = ((uint64_t)(uint32_t)rem_hi << 32 | rem_lo) - ((uint64_t)step_hi << 32 | step_lo);
    rem_lo = (uint32_t)m, rem_hi = (int)(uint32_t)(m >> 32);
    return r;
  }
};

// 16 (or 4) bytes of every lane into LDS at `lds` + lane * 16 (4); counted by vmcnt.  The
// scalar write of M0 needs one wait state before the load.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16(uint32_t lds, int4v r, uint32_t off) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(off), "s"(r), "s"(lds)
               : "memory", "m0");
}
__device__ __forceinline__ void copy4(uint32_t lds, int4v r, uint32_t off) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(off), "s"(r), "s"(lds)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// All but OPEN of this wave's copies have landed and its reads are done; then all waves' are.
template <int OPEN>
__device__ __forceinline__ void part_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(OPEN) : "memory");
}

// One operand: R rows (of A or columns of B) a tile, WT of them a wave.
// PACK (B, where C has 16 bits): the columns are spread over the fragments so that a lane's
// accumulators of two fragments are eight neighbouring columns, one 16-byte store.
template <class T, bool KC, int R, int WT, int WAVES, bool PACK = false>
struct PipeOperand {
  static constexpr int BYTES = R * kRowBytes;  // of a slot, either order
  static constexpr int COPIES = R / 8 / WAVES;
  static constexpr int SUB = WT / 16;
  static constexpr int READ = KC || T::BYTES != 4 ? 1 : SUB >= 4 ? 4 : 2;  // see read()
  static_assert(SUB % READ == 0, "whole groups of columns");
  static constexpr bool PACKED = PACK;
  static_assert(!PACK || (READ == 1 && SUB % 2 == 0), "pairs of fragments");
  static constexpr int KS = kRowBytes / T::BYTES;
  static constexpr int K_ROW = R * T::BYTES;   // bytes of a k row (rows contiguous)
  static_assert(COPIES * WAVES * 8 == R, "whole copies");
  static_assert(KC || T::BYTES == 4 || R >= 64, "f(k) needs four positions");
  static __device__ __forceinline__ int swizzle(int k) {
    if constexpr (R >= 128) return (k & 3) | ((k >> 3) & 1) << 2;
    return ((k >> 1) & 1) | ((k >> 3) & 1) << 1;  // two k rows share the 256 bytes of the banks
  }

  uint32_t off[COPIES];  // of this lane's 16 bytes from the tile's first
  const char* base;
  int64_t left;          // bytes of the operand from `base` on
  int64_t step;          // bytes a K step moves by
  uint32_t lane_at[KC ? 2 : T::BYTES == 4 ? 1 : SUB];  // fragment reads, from the slot

  // first: the tile's first row; rows: of the operand that may be read; k_len: of the contraction
  __device__ __forceinline__ void init(const char* p, int64_t ld, int first, int rows, int k_len,
                                       int wave, int lane, int w0) {
    const int64_t ldb = ld * T::BYTES;
    if constexpr (KC) {
      base = p + (int64_t)first * ldb;
      left = (int64_t)(rows - first - 1) * ldb + (int64_t)k_len * T::BYTES;
      step = kRowBytes;
    } else {
      base = p + (int64_t)first * T::BYTES;
      left = (int64_t)(k_len - 1) * ldb + (int64_t)(rows - first) * T::BYTES;
      step = KS * ldb;
    }
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      int row, at;
      place_of(wave + i * WAVES, lane, row, at);
      off[i] = (uint32_t)(row * ldb) + (uint32_t)at;
    }
    const int l16 = lane & 15, g = lane >> 4;
    if constexpr (KC) {
      const int r = w0 + row_of(0, l16), sw = place(r);
      lane_at[0] = (uint32_t)(r * kRowBytes + ((g ^ sw) << 4));
      lane_at[1] = (uint32_t)(r * kRowBytes + (((g + 4) ^ sw) << 4));
    } else if constexpr (T::BYTES == 4) {
      lane_at[0] = (uint32_t)(4 * g * K_ROW + (w0 + READ * l16) * 4);
    } else {
      const int k = 8 * g + (l16 >> 2), f = swizzle(k);
#pragma unroll
      for (int j = 0; j < SUB; ++j)
      {
        // lane l16 fetches columns row_of(j, 4 (l16 mod 4)) .. + 3 of its k row
        const int c = w0 + row_of(j, 4 * (l16 & 3));
        lane_at[j] = (uint32_t)(k * K_ROW + (((c >> 4) ^ f) << 5) + (c & 15) * 2);
      }
    }
  }

  // Which row (k contiguous) or k row, and which byte of it in the step, lane `lane` of copy j
  // moves.
  static __device__ __forceinline__ void place_of(int j, int lane, int& row, int& at) {
    if constexpr (KC) {
      row = j * 8 + lane / 8;
      at = ((lane & 7) ^ place(row)) * 16;
    } else {
      const int b = j * 1024 + lane * 16, in = b % K_ROW;
      row = b / K_ROW;
      at = T::BYTES == 4 ? in : ((((in >> 5) ^ swizzle(row)) << 5) | (in & 31));
    }
  }
  __device__ __forceinline__ int4v words(int kt) const {
    return buffer_words(base + kt * step, left - kt * step);
  }
  __device__ __forceinline__ void start(Walk& walk) const { walk.init(base, left, step); }
  __device__ __forceinline__ void copy(int i, int4v r, uint32_t lds, int wave) const {
    copy16(__builtin_amdgcn_readfirstlane(lds + (uint32_t)(wave + i * WAVES) * 1024u), r, off[i]);
  }
  __device__ __forceinline__ void issue(int kt, uint32_t lds, int wave) const {
    const int4v r = words(kt);
#pragma unroll
    for (int i = 0; i < COPIES; ++i) copy(i, r, lds, wave);
  }

  // Both halves of a K step, 16 bytes of k a lane each, for fragment i (of 16 rows), or for
  // the READ fragments from i on where a lane reads several columns at once.
  __device__ __forceinline__ void read(const char* slot, int i, int8v* f) const {
    if constexpr (KC) {
      // (the same place in every fragment: place() has row_of(i, 0)'s bits out)
      f[0] = both(*(const int4v*)(slot + lane_at[0] + row_of(i, 0) * kRowBytes),
                  *(const int4v*)(slot + lane_at[1] + row_of(i, 0) * kRowBytes));
    } else if constexpr (T::BYTES == 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const char* at = slot + lane_at[0] + q * K_ROW + 64 * i;
        typedef int group __attribute__((ext_vector_type(READ)));
        const group u = *(const group*)at, v = *(const group*)(at + 16 * K_ROW);
#pragma unroll
        for (int x = 0; x < READ; ++x) {
          f[x][q] = u[x];
          f[x][4 + q] = v[x];
        }
      }
    } else {
      f[0] = both(turned(slot + lane_at[i]), turned(slot + lane_at[i] + 32 * K_ROW));
    }
  }
  static __device__ __forceinline__ int8v both(int4v lo, int4v hi) {
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ int4v turned(const char* at) {
    typedef __attribute__((address_space(3))) short4v lds_short4;
    const short4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(lds_char*)at);
    const short4v b =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(lds_char*)(at + 4 * K_ROW));
    return __builtin_bit_cast(int4v, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  // The row that fragment i's row x of the wave's is.
  static __device__ __forceinline__ int row_of(int i, int x) {
    if constexpr (PACK) return 32 * (i >> 1) + 8 * (x >> 2) + 4 * (i & 1) + (x & 3);
    return 16 * (i - i % READ) + READ * x + i % READ;
  }
  // Where k is contiguous: the 16-byte group c of row r lies at c ^ place(r).  The 16 rows of a
  // fragment at one c then fall into 16 different groups of banks (two rows share 256 bytes).
  static __device__ __forceinline__ int place(int r) {
    if constexpr (PACK) return ((r >> 1) & 1) | ((r >> 3) & 3) << 1;
    return (r >> 1) & 7;
  }
  // The last K step holds k_bytes of each row: clear the rest, which came from beyond the row.
  static __device__ __forceinline__ void clear_tail(char* slot, int k_bytes, int tid, int threads) {
    for (int t = tid; t < R * 8; t += threads) {
      const int row = t >> 3, c = t & 7, n = k_bytes - 16 * c;
      if (n >= 16) continue;
      int4v* at = (int4v*)(slot + row * kRowBytes + ((c ^ place(row)) << 4));
      int4v v = {0, 0, 0, 0};
      if (n > 0) {
        v = *at;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int m = n - 4 * w;
          if (m <= 0) v[w] = 0;
          else if (m < 4) v[w] &= (int)((1u << (8 * m)) - 1u);
        }
      }
      *at = v;
    }
  }
};

__device__ __forceinline__ int4v half_of(int8v f, int h) {
  return h ? __builtin_shufflevector(f, f, 4, 5, 6, 7) : __builtin_shufflevector(f, f, 0, 1, 2, 3);
}

// 16 bytes at p of any alignment, of which the first n bytes (whole elements) may be read; the
// others are zero.
template <class T>
__device__ __forceinline__ int4v load_group(const char* p, int64_t n) {
  constexpr int PER = 16 / T::BYTES;
  int4v v = {0, 0, 0, 0};
  if (n >= 16) {
    __builtin_memcpy(&v, p, 16);
  } else if (n > 0) {
    typename T::type e[PER] = {};
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * T::BYTES < n) __builtin_memcpy(e + i, p + i * T::BYTES, T::BYTES);
    __builtin_memcpy(&v, e, 16);
  }
  return v;
}

// The copies of an operand of any alignment and leading dimension, through registers: the
// same groups at the same places as PipeOperand's.
template <class T, class O, bool KC, int WAVES>
struct StagedCopy {
  int4v v[O::COPIES];
  const char* base;
  int64_t off[O::COPIES];
  int64_t left, step;
  int k_of[O::COPIES];  // KC: the group's first byte of k in a step; else its k row
  int inside;           // KC: bit i: group i's row is one of the operand's
  int64_t k_len;        // KC: bytes of k; else k rows

  __device__ __forceinline__ void init(const char* p, int64_t ld, int first, int rows, int k,
                                       int wave, int lane) {
    const int64_t ldb = ld * T::BYTES;
    base = p + (KC ? (int64_t)first * ldb : (int64_t)first * T::BYTES);
    left = (int64_t)(k - 1) * ldb + (int64_t)(rows - first) * T::BYTES;  // (not KC)
    step = KC ? kRowBytes : O::KS * ldb;
    k_len = KC ? (int64_t)k * T::BYTES : k;
    inside = 0;
#pragma unroll
    for (int i = 0; i < O::COPIES; ++i) {
      int row, at;
      O::place_of(wave + i * WAVES, lane, row, at);
      off[i] = row * ldb + at;
      k_of[i] = KC ? at : row;
      if (first + row < rows) inside |= 1 << i;
    }
  }
  __device__ __forceinline__ void load(int kt) {
#pragma unroll
    for (int i = 0; i < O::COPIES; ++i) {
      int64_t n;  // bytes that may be read
      if constexpr (KC)
        n = inside >> i & 1 ? k_len - (int64_t)kt * kRowBytes - k_of[i] : 0;
      else  // past the last column a group holds the next row's values, which go nowhere
        n = kt * O::KS + k_of[i] < k_len ? left - kt * step - off[i] : 0;
      v[i] = load_group<T>(base + kt * step + off[i], n);
    }
  }
  __device__ __forceinline__ void store(char* part, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < O::COPIES; ++i)
      *(int4v*)(part + (wave + i * WAVES) * 1024 + lane * 16) = v[i];
  }
};

// 16 bytes of k a lane from each side.
template <class T>
__device__ __forceinline__ float4v mma_half(int4v a, int4v b, float4v c) {
  if constexpr (T::CODE == GEMM_LP_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf168v, a),
                                                   __builtin_bit_cast(bf168v, b), c, 0, 0, 0);
  } else if constexpr (T::CODE == GEMM_LP_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, a),
                                                  __builtin_bit_cast(half8v, b), c, 0, 0, 0);
  } else {
    const float4v x = __builtin_bit_cast(float4v, a), y = __builtin_bit_cast(float4v, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
  }
}

// What one workgroup computes: C's rows m0 .. m_end and columns n0 .. from A's and B's rows.
struct TileOf {
  const char* A;
  const char* B;
  int64_t c_base;
  int m0, m_end, n0, e, k_end;
  bool half;
};
template <class T, bool WGRAD, int BM, int BN, int HALF = 0>
__device__ __forceinline__ bool locate(const LpArgs& p, TileOf& w) {
  w.A = (const char*)p.A;
  w.B = (const char*)p.B;
  w.c_base = 0;
  if constexpr (WGRAD) {
    const int tiles_m = (p.M + BM - 1) / BM, per = tiles_m * p.tiles_n;
    int tm, tn;
    wgrad_tile(blockIdx.x, per, tiles_m, p.tiles_n, w.e, tm, tn);
    const int lo = clamped_offset(p.offsets, w.e, p.rows);
    const int hi = clamped_offset(p.offsets, w.e + 1, p.rows);
    w.A += (int64_t)lo * p.lda * T::BYTES;
    w.B += (int64_t)lo * p.ldb * T::BYTES;
    w.k_end = max(hi - lo, 0);
    w.m0 = tm * BM;
    w.m_end = p.M;
    w.n0 = tn * BN;
    w.c_base = w.e * p.stride_c;
  } else {
    TileAt t;
    if (!find_tile<BM, HALF>(p, blockIdx.x, gridDim.x, t)) return false;
    w.e = __builtin_amdgcn_readfirstlane(t.e);
    w.half = __builtin_amdgcn_readfirstlane((int)t.half) != 0;
    w.k_end = w.e < 0 ? 0 : p.K;
    if (w.e > 0) w.B += w.e * p.stride_b * T::BYTES;
    w.m0 = __builtin_amdgcn_readfirstlane(t.row0);
    w.m_end = __builtin_amdgcn_readfirstlane(t.row_end);
    w.n0 = __builtin_amdgcn_readfirstlane(t.tn) * BN;
  }
  return true;
}

// How 8-bit values are scaled: FP32 scales, B's column by column or by blocks of 128 columns; or
// powers of two, one exponent byte for each row and column.
enum { kScaleRows = 0, kScaleBlocks = 1, kScaleExponents = 2 };

// The copies of a K step's scales (8-bit values) into the slot's table, A's rows first: FP32
// numbers, 64 a wave, or exponent bytes, which every wave copies for A or for B (the same bytes:
// a wave's copies of a step then have one count).
template <int HOW, int BM, int BN>
struct ScaleCopy {
  static constexpr bool EXP = HOW == kScaleExponents;
  static constexpr int B_AT = EXP ? 256 : BM * 4;       // B's part
  static constexpr int BYTES = EXP ? 512 : (BM + BN) * 4;
  static constexpr int WAVES = EXP ? 64 : (BM + BN) / 64;  // waves that copy
  static_assert(!EXP || (BM <= 256 && BN <= 256), "64 words an operand");
  const char* base;
  int64_t left, step;
  uint32_t off;
  uint32_t to;
  __device__ __forceinline__ void init(const LpArgs& p, const TileOf& w, int steps, int wave,
                                       int lane) {
    if constexpr (EXP) {
      const bool b = wave & 1;
      step = b ? p.ldsb : p.ldsa;
      base = (const char*)(b ? p.SB : p.SA) + (b ? w.n0 : w.m0);
      left = (int64_t)(steps - 1) * step + (b ? p.N - w.n0 : w.m_end - w.m0);
      off = (uint32_t)lane * 4;
      to = b ? B_AT : 0;
      return;
    }
    const int r = wave * 64 + lane;
    step = 4;
    to = (uint32_t)wave * 256;
    if (wave < BM / 64) {
      const int rows = w.m_end - w.m0;
      base = (const char*)(p.SA + (int64_t)w.m0 * p.ldsa);
      off = (uint32_t)(min(r, rows - 1) * p.ldsa * 4);
      left = ((int64_t)(rows - 1) * p.ldsa + steps) * 4;
    } else {
      const int first = w.n0 >> p.sb_shift;
      const int n = min(w.n0 + r - BM, p.N - 1) >> p.sb_shift;
      base = (const char*)(p.SB + w.e * p.stride_sb + (int64_t)first * p.ldsb);
      off = (uint32_t)((n - first) * p.ldsb * 4);
      left = ((int64_t)(((p.N - 1) >> p.sb_shift) - first) * p.ldsb + steps) * 4;
    }
  }
  __device__ __forceinline__ int4v words(int kt) const {
    return buffer_words(base + kt * step, left - kt * step);
  }
  __device__ __forceinline__ void copy(int4v r, uint32_t table) const {
    copy4(__builtin_amdgcn_readfirstlane(table + to), r, off);
  }
  __device__ __forceinline__ void issue(int kt, uint32_t table) const { copy(words(kt), table); }

  // Scales from the table: of row r of A, of column c of B, of columns c .. c + 3.
  static __device__ __forceinline__ float number(uint32_t byte) {
    return __builtin_bit_cast(float, byte << 23);  // 2^(byte - 127)
  }
  static __device__ __forceinline__ float a(const char* table, int r) {
    if constexpr (EXP) return number((uint8_t)table[r]);
    return ((const float*)table)[r];
  }
  static __device__ __forceinline__ float b(const char* table, int c) {
    if constexpr (EXP) return number((uint8_t)table[B_AT + c]);
    return ((const float*)(table + B_AT))[c];
  }
  static __device__ __forceinline__ float4v b4(const char* table, int c) {
    if constexpr (EXP) {
      const uint32_t x = *(const uint32_t*)(table + B_AT + c);
      return float4v{number(x & 255), number(x >> 8 & 255), number(x >> 16 & 255), number(x >> 24)};
    }
    return *(const float4v*)(table + B_AT + 4 * c);
  }
};

// One wave's accumulators into C.  m: C's row of fragment i for this lane.
template <class OB, int OUT, int SM, int SN, class F>
__device__ __forceinline__ void store_tile(const LpArgs& p, const TileOf& w, int wn, int g,
                                           const float4v (&acc)[SM][SN], F row) {
#pragma unroll
  for (int i = 0; i < SM; ++i) {
    const int m = row(i);
    if (m >= w.m_end) continue;
    const int64_t at = w.c_base + (int64_t)m * p.ldc;
    if constexpr (OB::PACKED) {
#pragma unroll
      for (int j = 0; j < SN; j += 2) {
        const int n = w.n0 + wn + 16 * j + 8 * g;
        float v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = acc[i][j + x / 4][x % 4];
        store_row<8, OUT>(p.C, at + n, p.N - n, p.c_type, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < SN; ++j) {
        // of READ fragments from j0 on, a lane has 4 READ neighbouring columns, fragment by
        // fragment in each register: the j - j0 th four of them
        constexpr int READ = OB::READ;
        const int q = j % READ, j0 = j - q;
        float v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = acc[i][j0 + (4 * q + x) % READ][(4 * q + x) / READ];
        const int n = w.n0 + wn + 16 * j0 + 4 * READ * g + 4 * q;
        store_row<4, OUT>(p.C, at + n, p.N - n, p.c_type, v);
      }
    }
  }
}

// STAGED: operands of any alignment, through registers.
// KG: groups of waves that share the tile, each with slots of its own and every KG-th K step;
// they add their sums through LDS in a fixed order.  With fewer tiles than CUs one group would
// wait for memory most of the time.
template <class T, bool AKC, bool BKC, bool WGRAD, int BM, int BN, int WM, int WN, int HOW,
          bool STAGED, int KG>
__global__ __launch_bounds__(WM * WN * 64 * KG, BM == 64 ? 4 : 2) void lp_pipe_kernel(LpArgs p) {
  constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
  constexpr int WTM = BM / WM, WTN = BN / WN, SM = WTM / 16, SN = WTN / 16;
  constexpr bool F8T = T::BYTES == 1;
  using OA = PipeOperand<T, AKC, BM, WTM, WAVES>;
  constexpr bool PACK = T::BYTES == 2;  // (C has 16 bits)
  using OB = PipeOperand<T, BKC, BN, WTN, WAVES, PACK>;
  using OS = ScaleCopy<HOW, BM, BN>;
  constexpr int SCALES = F8T ? OS::BYTES : 0;
  constexpr int SLOT = OA::BYTES + OB::BYTES + SCALES;
  __shared__ __align__(1024) char all_lds[KG * 2 * SLOT];
  const int group = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / THREADS);
  char* lds = all_lds + group * 2 * SLOT;
  const int tid = KG == 1 ? threadIdx.x : threadIdx.x % THREADS, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;

  TileOf w;
  // A tile of FP32 rows takes the matrix cores long enough for half of it to be worth leaving
  // out: each wave then has the first half of its fragments, from half as far down (2048 rows of
  // 8 experts, warm: X W 2048 -> 1024 97 us, 108 in whole tiles; 1024 -> 2048 85, 92; X W^T 91,
  // 104; 84, 91).
  constexpr int HALF = T::BYTES == 4 && !WGRAD && BM == 64 && SM == 2 ? BM / 2 : 0;
  if (!locate<T, WGRAD, BM, BN, HALF>(p, w)) return;
  const bool half = HALF > 0 && w.half;
  const int wm = (wave / WN) * (half ? WTM / 2 : WTM), wn = (wave % WN) * WTN;

  float4v acc[SM][SN] = {};
  const int steps = (w.k_end + OA::KS - 1) / OA::KS;
  if (steps > 0) {
    OA oa;
    OB ob;
    oa.init(w.A, p.lda, w.m0, w.m_end, w.k_end, wave, lane, wm);
    ob.init(w.B, p.ldb, w.n0, p.N, w.k_end, wave, lane, wn);
    const uint32_t lds0 =
        __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_char*)lds);
    OS os;
    if constexpr (F8T) os.init(p, w, steps, wave, lane);
    StagedCopy<T, OA, AKC, WAVES> ca;
    StagedCopy<T, OB, BKC, WAVES> cb;
    if constexpr (STAGED) {
      ca.init(w.A, p.lda, w.m0, w.m_end, w.k_end, wave, lane);
      cb.init(w.B, p.ldb, w.n0, p.N, w.k_end, wave, lane);
    }
    auto issue = [&](int kt, int slot) {
      const uint32_t at = lds0 + (uint32_t)(slot * SLOT);
      if constexpr (STAGED) {
        ca.load(kt);
        cb.load(kt);
      } else {
        oa.issue(kt, at, wave);
        ob.issue(kt, at + OA::BYTES, wave);
      }
      if constexpr (F8T) {
        static_assert(OS::EXP || OS::WAVES <= WAVES, "a wave copies 64 scales");
        if (wave < OS::WAVES) os.issue(kt, at + OA::BYTES + OB::BYTES);
      }
    };
    const int tail = (w.k_end % OA::KS) * T::BYTES;  // bytes of k in the last step, 0: all

    auto settle = [&](int slot) {  // what issue() left in registers
      if constexpr (STAGED) {
        ca.store(lds + slot * SLOT, wave, lane);
        cb.store(lds + slot * SLOT + OA::BYTES, wave, lane);
      }
    };

    if (group < steps) {
      issue(group, 0);
      settle(0);
    }
    // 8-bit values: the next step's copies go out between this one's products, since a wave waits
    // for each to be taken (8192 x 4096 x 4096: 237 us, 260 with the copies first; 263 and 265
    // with a scale for each column, 258 and 264 with exponents); past the last step they have
    // nothing to copy, zeros into a slot that is not read again.  The others, whose steps are
    // shorter, lose by it (bf16 X W^T 1167 us, 1024 with the copies first).
    constexpr bool SPREAD = F8T && !STAGED && KG == 1 && BM >= 128;
    constexpr int SENT = OA::COPIES + OB::COPIES + 1;
    static_assert(!SPREAD || OS::EXP || OS::WAVES == WAVES, "every wave copies scales");
    const int rounds = (steps + KG - 1) / KG;
    auto loop = [&](auto fragments) {  // of A a wave
      for (int it = 0; it < rounds; ++it) {
        const int kt = it * KG + group;
        part_barrier<0>();
        int4v ra, rb, rs;
        int sent = 0;  // (a constant wherever it is used)
        const uint32_t to = lds0 + (uint32_t)(((it + 1) & 1) * SLOT);
        if constexpr (SPREAD) {
          ra = oa.words(kt + 1);
          rb = ob.words(kt + 1);
          rs = os.words(kt + 1);
          const bool more = kt + 1 < steps;
          ra[2] = more ? ra[2] : 0;
          rb[2] = more ? rb[2] : 0;
          rs[2] = more ? rs[2] : 0;
        } else {
          if (kt + KG < steps) issue(kt + KG, (it + 1) & 1);
        }
        auto send = [&](int product, int products) {  // behind this product of so many
          if constexpr (SPREAD) {
            while (sent * products < (product + 1) * SENT && sent < SENT) {
              if (sent < OB::COPIES) ob.copy(sent, rb, to + OA::BYTES, wave);
              else if (sent < OB::COPIES + OA::COPIES) oa.copy(sent - OB::COPIES, ra, to, wave);
              else os.copy(rs, to + OA::BYTES + OB::BYTES);
              ++sent;
            }
          }
        };
        char* sa = lds + (it & 1) * SLOT;
        char* sb = sa + OA::BYTES;
        if (!STAGED && (AKC || BKC) && tail != 0 && it + 1 == rounds) {
          if (KG == 1 || kt + 1 == steps) {
            if constexpr (AKC) OA::clear_tail(sa, tail, tid, THREADS);
            if constexpr (BKC) OB::clear_tail(sb, tail, tid, THREADS);
          }
          __syncthreads();
        }
        if (KG > 1 && kt >= steps) continue;
        if constexpr (!F8T) {
          constexpr int N = decltype(fragments)::value;
          int8v a[SM], b[SN];
#pragma unroll
          for (int j = 0; j < SN; j += OB::READ) ob.read(sb, j, b + j);
#pragma unroll
          for (int i = 0; i < N; i += OA::READ) oa.read(sa, i, a + i);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
              for (int j = 0; j < SN; ++j)
                acc[i][j] = mma_half<T>(half_of(b[j], h), half_of(a[i], h), acc[i][j]);
        } else {
          const char* table = sb + OB::BYTES;
          int8v b[SN], a[2];
#pragma unroll
          for (int j = 0; j < SN; ++j) ob.read(sb, j, b + j);
          oa.read(sa, 0, a);
          float4v s_b[SN];
          float s_a[SM];
#pragma unroll
          for (int i = 0; i < SM; ++i) s_a[i] = OS::a(table, wm + 16 * i + l16);
          if constexpr (HOW == kScaleBlocks) {
            // the wave's columns lie in one block of 128: one factor a row
            static_assert(kBlock % WTN == 0, "a wave's columns cross a block of scales");
            const float block = OS::b(table, wn);
#pragma unroll
            for (int i = 0; i < SM; ++i) s_a[i] *= block;
          } else {
#pragma unroll
            for (int j = 0; j < SN; ++j) s_b[j] = OS::b4(table, wn + OB::row_of(j, 4 * g));
          }
          // The sums of a step are scaled and added kLag products behind, while the matrix
          // cores work on the next ones.
          constexpr int kLag = 1, kRing = kLag + 1;
          float4v d[kRing];
#pragma unroll
          for (int s = 0; s < SM * SN + kLag; ++s) {
            if (s < SM * SN) {
              const int i = s / SN, j = s % SN;
              if (j == 0 && i + 1 < SM) oa.read(sa, i + 1, a + ((i + 1) & 1));
              const float4v z = {0.0f, 0.0f, 0.0f, 0.0f};
              d[s % kRing] = mma_fp8_step(half_of(b[j], 0), half_of(b[j], 1), half_of(a[i & 1], 0),
                                          half_of(a[i & 1], 1), z);
              send(s, SM * SN * 3 / 4);  // the last with a quarter of the step to land
            }
            if (s >= kLag) {
              const int i = (s - kLag) / SN, j = (s - kLag) % SN;
              const float4v v = d[(s - kLag) % kRing];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                if constexpr (HOW == kScaleBlocks)
                  acc[i][j][r] += v[r] * s_a[i];
                else
                  acc[i][j][r] += v[r] * (s_a[i] * s_b[j][r]);
              }
            }
          }
        }
        if (kt + KG < steps) settle((it + 1) & 1);
      }
    };
    if constexpr (HALF > 0) {
      if (half) loop(std::integral_constant<int, SM / 2>{});
      else loop(std::integral_constant<int, SM>{});
    } else {
      loop(std::integral_constant<int, SM>{});
    }
    if constexpr (KG > 1) {
      // the groups' sums, in their order: lane by lane, 16 bytes at a time
      static_assert(SM * SN * 16 * THREADS <= 2 * SLOT, "a group's sums in its slots");
      __syncthreads();
      if (group > 0) {
#pragma unroll
        for (int i = 0; i < SM; ++i)
#pragma unroll
          for (int j = 0; j < SN; ++j)
            *(float4v*)(lds + ((i * SN + j) * THREADS + tid) * 16) = acc[i][j];
      }
      __syncthreads();
      if (group > 0) return;
#pragma unroll
      for (int o = 1; o < KG; ++o)
#pragma unroll
        for (int i = 0; i < SM; ++i)
#pragma unroll
          for (int j = 0; j < SN; ++j)
            acc[i][j] += *(const float4v*)(lds + o * 2 * SLOT + ((i * SN + j) * THREADS + tid) * 16);
    }
  }
  if (KG > 1 && group > 0) return;

  constexpr int OUT = F8T ? -1 : T::CODE;
  store_tile<OB, OUT>(p, w, wn, g, acc,
                     [&](int i) {
                       return half && i >= SM / 2 ? w.m_end : w.m0 + wm + OA::row_of(i, l16);
                     });
}

}  // namespace gemmlp
