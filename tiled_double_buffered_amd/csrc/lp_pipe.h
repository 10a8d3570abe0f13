// The product kernel for operands whose rows start at multiples of 4 bytes: tiles go from
// memory straight into LDS (gfx950's direct-to-LDS loads), two slots in turn, one barrier a
// K step.
//
// A K step is 128 bytes of every row where k is contiguous (128 8-bit, 64 16-bit, 32 32-bit
// values), so that all types share one LDS layout:
//   k contiguous: rows of 128 bytes; the 16-byte group c of row r lies at c ^ (r / 2 mod 8),
//     so that the 16 rows a fragment reads at one c fall into 16 different groups of banks;
//   rows contiguous (the operand's k is the slow axis), 16-bit: k rows of R values, read
//     through the transposing LDS load, which hands each lane four k of one column; the 32
//     bytes of 16 columns at position j lie at j ^ f(k), f(k) = k mod 4 + 4 (k / 8 mod 2), so
//     that the eight k rows that half a wave reads fall into different banks;
//   rows contiguous, 32-bit: k rows of R values as they are; a lane reads four neighbouring
//     columns of one k, which are four 16-column fragments, column 4 i + q the i-th of the
//     q-th, and the epilogue undoes that order.
// The copies write LDS in lane order, so each lane fetches what belongs at its place.
//
// Accumulators are transposed (D's rows are columns of C): a lane holds four neighbouring
// columns of one row of C and stores them at once.
#pragma once

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

// This wave's copies have landed and its reads are done; then all waves' are.
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// One operand: R rows (of A or columns of B) a tile, WT of them a wave.
template <class T, bool KC, int R, int WT, int WAVES>
struct PipeOperand {
  static constexpr int BYTES = R * kRowBytes;  // of a slot, either order
  static constexpr int COPIES = R / 8 / WAVES;
  static constexpr int SUB = WT / 16;
  static constexpr int KS = kRowBytes / T::BYTES;
  static constexpr int K_ROW = R * T::BYTES;   // bytes of a k row (rows contiguous)
  static_assert(COPIES * WAVES * 8 == R, "whole copies");
  static_assert(KC || T::BYTES == 4 || R >= 128, "f(k) needs eight positions");

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
      const int j = wave + i * WAVES;
      if constexpr (KC) {
        const int row = j * 8 + lane / 8;
        off[i] = (uint32_t)(row * ldb) + (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 16);
      } else {
        const int at = j * 1024 + lane * 16, k = at / K_ROW, in = at % K_ROW;
        if constexpr (T::BYTES == 4)
          off[i] = (uint32_t)(k * ldb) + (uint32_t)in;
        else
          off[i] = (uint32_t)(k * ldb) +
                   (uint32_t)((((in >> 5) ^ ((k & 3) | ((k >> 3) & 1) << 2)) << 5) | (in & 31));
      }
    }
    const int l16 = lane & 15, g = lane >> 4;
    if constexpr (KC) {
      const int sw = (l16 >> 1) & 7;
      lane_at[0] = (uint32_t)((w0 + l16) * kRowBytes + ((g ^ sw) << 4));
      lane_at[1] = (uint32_t)((w0 + l16) * kRowBytes + (((g + 4) ^ sw) << 4));
    } else if constexpr (T::BYTES == 4) {
      lane_at[0] = (uint32_t)(4 * g * K_ROW + (w0 + 4 * l16) * 4);
    } else {
      const int k = 8 * g + (l16 >> 2), f = (k & 3) | ((k >> 3) & 1) << 2;
#pragma unroll
      for (int j = 0; j < SUB; ++j)
        lane_at[j] = (uint32_t)(k * K_ROW + ((((w0 >> 4) + j) ^ f) << 5) + (l16 & 3) * 8);
    }
  }

  __device__ __forceinline__ void issue(int kt, uint32_t lds, int wave) const {
    const int4v r = buffer_words(base + kt * step, left - kt * step);
#pragma unroll
    for (int i = 0; i < COPIES; ++i)
      copy16(__builtin_amdgcn_readfirstlane(lds + (uint32_t)(wave + i * WAVES) * 1024u), r, off[i]);
  }

  // Half h of a K step: 16 bytes of k a lane for each 16-row fragment.
  __device__ __forceinline__ void read(const char* slot, int h, int4v* f) const {
    if constexpr (KC) {
#pragma unroll
      for (int i = 0; i < SUB; ++i)
        f[i] = *(const int4v*)(slot + lane_at[h] + i * 16 * kRowBytes);
    } else if constexpr (T::BYTES == 4) {
#pragma unroll
      for (int j = 0; j < SUB / 4; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int4v v = *(const int4v*)(slot + lane_at[0] + (16 * h + q) * K_ROW + 256 * j);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[4 * j + i][q] = v[i];
        }
    } else {
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        const char* at = slot + lane_at[j] + h * 32 * K_ROW;
        typedef __attribute__((address_space(3))) short4v lds_short4;
        const short4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(lds_char*)at);
        const short4v b =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(lds_char*)(at + 4 * K_ROW));
        f[j] = __builtin_bit_cast(int4v, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  }
  // The row that fragment i's row x of the wave's is.
  static __device__ __forceinline__ int row_of(int i, int x) {
    if constexpr (!KC && T::BYTES == 4) return 64 * (i >> 2) + 4 * x + (i & 3);
    return 16 * i + x;
  }
  // The last K step holds k_bytes of each row: clear the rest, which came from beyond the row.
  static __device__ __forceinline__ void clear_tail(char* slot, int k_bytes, int tid, int threads) {
    for (int t = tid; t < R * 8; t += threads) {
      const int row = t >> 3, c = t & 7, n = k_bytes - 16 * c;
      if (n >= 16) continue;
      int4v* at = (int4v*)(slot + row * kRowBytes + ((c ^ ((row >> 1) & 7)) << 4));
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

// FAST8: 8-bit values through the 8-bit instruction; otherwise through the 16-bit one.
template <class T, bool AKC, bool BKC, bool WGRAD, int BM, int BN, int WM, int WN, bool FAST8>
__global__ __launch_bounds__(WM * WN * 64) void lp_pipe_kernel(LpArgs p) {
  constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
  constexpr int WTM = BM / WM, WTN = BN / WN, SM = WTM / 16, SN = WTN / 16;
  constexpr bool F8T = T::BYTES == 1;
  using OA = PipeOperand<T, AKC, BM, WTM, WAVES>;
  using OB = PipeOperand<T, BKC, BN, WTN, WAVES>;
  constexpr int SCALES = F8T ? (BM + BN) * 4 : 0;
  constexpr int SLOT = OA::BYTES + OB::BYTES + SCALES;
  __shared__ __align__(1024) char lds[2 * SLOT];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;

  const char* A = (const char*)p.A;
  const char* B = (const char*)p.B;
  int64_t c_base = 0;
  int m0, m_end, n0, e, k_end, a_rows;
  if constexpr (WGRAD) {
    const int tiles_m = (p.M + BM - 1) / BM, per = tiles_m * p.tiles_n;
    const int id = xcd_order(blockIdx.x, gridDim.x);
    e = id / per;
    int tm, tn;
    band_order(id - e * per, tiles_m, p.tiles_n, tm, tn);
    const int lo = clamped_offset(p.offsets, e, p.rows);
    const int hi = clamped_offset(p.offsets, e + 1, p.rows);
    A += (int64_t)lo * p.lda * T::BYTES;
    B += (int64_t)lo * p.ldb * T::BYTES;
    k_end = max(hi - lo, 0);
    m0 = tm * BM;
    m_end = a_rows = p.M;
    n0 = tn * BN;
    c_base = e * p.stride_c;
  } else {
    TileAt t;
    if (!find_tile(p, BM, blockIdx.x, gridDim.x, t)) return;
    e = __builtin_amdgcn_readfirstlane(t.e);
    k_end = e < 0 ? 0 : p.K;
    if (e > 0) B += e * p.stride_b * T::BYTES;
    m0 = __builtin_amdgcn_readfirstlane(t.row0);
    m_end = __builtin_amdgcn_readfirstlane(t.row_end);
    n0 = __builtin_amdgcn_readfirstlane(t.tn) * BN;
    a_rows = m_end;
  }
  const int wm = (wave / WN) * WTM, wn = (wave % WN) * WTN;

  float4v acc[SM][SN] = {};
  const int steps = (k_end + OA::KS - 1) / OA::KS;
  if (steps > 0) {
    OA oa;
    OB ob;
    oa.init(A, p.lda, m0, a_rows, k_end, wave, lane, wm);
    ob.init(B, p.ldb, n0, p.N, k_end, wave, lane, wn);
    const uint32_t lds0 =
        __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_char*)lds);
    // 8-bit: a K step's scales, one for each row of A and column of B, one copy of 64 a wave
    uint32_t s_off = 0;
    const char* s_base = nullptr;
    int64_t s_left = 0;
    constexpr int S_WAVES = (BM + BN) / 64;
    if constexpr (F8T) {
      static_assert(S_WAVES <= WAVES, "a wave copies 64 scales at most");
      const int r = wave * 64 + lane;
      if (wave < BM / 64) {
        s_base = (const char*)(p.SA + (int64_t)m0 * p.ldsa);
        const int rows = a_rows - m0;
        s_off = (uint32_t)(min(r, rows - 1) * p.ldsa * 4);
        s_left = ((int64_t)(rows - 1) * p.ldsa + steps) * 4;
      } else {
        const int n = min(n0 + r - BM, p.N - 1);
        s_base = (const char*)(p.SB + e * p.stride_sb + (int64_t)(n0 >> p.sb_shift) * p.ldsb);
        s_off = (uint32_t)(((n >> p.sb_shift) - (n0 >> p.sb_shift)) * p.ldsb * 4);
        s_left = ((int64_t)(((p.N - 1) >> p.sb_shift) - (n0 >> p.sb_shift)) * p.ldsb + steps) * 4;
      }
    }
    auto issue = [&](int kt, int slot) {
      const uint32_t at = lds0 + (uint32_t)(slot * SLOT);
      oa.issue(kt, at, wave);
      ob.issue(kt, at + OA::BYTES, wave);
      if constexpr (F8T) {
        if (wave < S_WAVES)
          copy4(__builtin_amdgcn_readfirstlane(at + OA::BYTES + OB::BYTES + (uint32_t)wave * 256u),
                buffer_words(s_base + kt * 4, s_left - kt * 4), s_off);
      }
    };
    const int tail = (k_end % OA::KS) * T::BYTES;  // bytes of k in the last step, 0: all

    issue(0, 0);
    for (int kt = 0; kt < steps; ++kt) {
      step_barrier();
      if (kt + 1 < steps) issue(kt + 1, (kt + 1) & 1);
      char* sa = lds + (kt & 1) * SLOT;
      char* sb = sa + OA::BYTES;
      if ((AKC || BKC) && tail != 0 && kt + 1 == steps) {
        if constexpr (AKC) OA::clear_tail(sa, tail, tid, THREADS);
        if constexpr (BKC) OB::clear_tail(sb, tail, tid, THREADS);
        __syncthreads();
      }
      if constexpr (!F8T) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int4v fa[SM], fb[SN];
          ob.read(sb, h, fb);
          oa.read(sa, h, fa);
#pragma unroll
          for (int i = 0; i < SM; ++i)
#pragma unroll
            for (int j = 0; j < SN; ++j) acc[i][j] = mma_half<T>(fb[j], fa[i], acc[i][j]);
        }
      } else {
        const float* scales = (const float*)(sb + OB::BYTES);
        int4v b0[SN], b1[SN];
        ob.read(sb, 0, b0);
        ob.read(sb, 1, b1);
        float4v s_b[SN];
#pragma unroll
        for (int j = 0; j < SN; ++j)
          s_b[j] = *(const float4v*)(scales + BM + wn + 16 * j + 4 * g);
#pragma unroll
        for (int i = 0; i < SM; ++i) {
          const int4v a0 = *(const int4v*)(sa + oa.lane_at[0] + i * 16 * kRowBytes);
          const int4v a1 = *(const int4v*)(sa + oa.lane_at[1] + i * 16 * kRowBytes);
          const float s_a = scales[wm + 16 * i + l16];
#pragma unroll
          for (int j = 0; j < SN; ++j) {
            const float4v z = {0.0f, 0.0f, 0.0f, 0.0f};
            float4v d;
            if constexpr (FAST8)
              d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                  __builtin_shufflevector(b0[j], b1[j], 0, 1, 2, 3, 4, 5, 6, 7),
                  __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7), z, 0, 0, 0, 0, 0, 0);
            else
              d = mma_step<T>(b0[j], b1[j], a0, a1, z);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][r] += d[r] * (s_a * s_b[j][r]);
          }
        }
      }
    }
  }

  const int cb = type_bytes(p.c_type);
  const bool vec = (((uintptr_t)p.C | (uintptr_t)(p.ldc * cb) | (uintptr_t)(c_base * cb)) &
                    (uintptr_t)(4 * cb - 1)) == 0;
#pragma unroll
  for (int i = 0; i < SM; ++i) {
    const int m = m0 + wm + OA::row_of(i, l16);
    if (m >= m_end) continue;
#pragma unroll
    for (int j = 0; j < SN; ++j) {
      if constexpr (!BKC && T::BYTES == 4) {
        // fragments 4 q .. 4 q + 3, register r: columns 64 q + 16 g + 4 r .. + 3
        const int q = j >> 2, r = j & 3, n = n0 + wn + 64 * q + 16 * g + 4 * r;
        const float4v v = {acc[i][4 * q][r], acc[i][4 * q + 1][r], acc[i][4 * q + 2][r],
                           acc[i][4 * q + 3][r]};
        store4(p.C, c_base + (int64_t)m * p.ldc + n, p.N - n, vec, p.c_type, v);
      } else {
        const int n = n0 + wn + 16 * j + 4 * g;
        store4(p.C, c_base + (int64_t)m * p.ldc + n, p.N - n, vec, p.c_type, acc[i][j]);
      }
    }
  }
}

}  // namespace gemmlp
