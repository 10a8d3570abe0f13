// The pipelined product kernel for large products: 256 x 256 tiles, eight waves of 128 x 64,
// two LDS slots refilled in halves, so that a copy has one and a half K steps to land.
//
// The kernel of lp_pipe.h starts a step's copies when the slot's last reader is done and needs
// them one step later, and waits for them (8 bits: 40 % of all wave cycles).  Here each slot has
// three parts that are freed at different times: B, which a wave holds in registers for the
// whole step, the upper half A1 of A's rows, which the step's first products read, and the
// lower half A2.  A step has two barriers:
//   middle (before the products of the last A1 fragment): B, A1 of this step are read by all
//     waves, A2 of this step has landed; the copies of B, A1 (and scales) two steps on start;
//   end (before the products of the last A2 fragment): A2 of this step is read, B and A1 of
//     the next have landed; the copies of A2 two steps on start, and the next step's first
//     fragments are read while this step's last products run.
// A tile of 128 rows or fewer leaves A2 and its products out.
// Copies complete in order, so a wave waits until no more are open than were started after the
// part it needs.
#pragma once

#include <type_traits>

#include "lp_pipe.h"

namespace gemmlp {

template <class T, bool AKC, bool BKC, bool WGRAD, int HOW>
__global__ __launch_bounds__(512) void lp_deep_kernel(LpArgs p) {
  constexpr int BM = 256, BN = 256, WN = 4, WAVES = 8;
  constexpr int WTM = 128, WTN = 64, HALF = WTM / 2, SM = 8, SN = 4, SH = SM / 2;
  constexpr bool F8T = T::BYTES == 1;
  static_assert(!F8T || !exact(HOW), "not enough registers");
  constexpr bool PACK = T::BYTES <= 2;  // C has 16 bits
  using OA = PipeOperand<T, AKC, BM / 2, HALF, WAVES>;
  using OB = PipeOperand<T, BKC, BN, WTN, WAVES, PACK>;
  using OS = ScaleCopy<HOW, BM, BN>;
  constexpr int SCALES = F8T ? OS::BYTES : 0;
  constexpr int A1 = 0, A2 = OA::BYTES, B0 = 2 * OA::BYTES, S0 = B0 + OB::BYTES;
  constexpr int SLOT = S0 + SCALES;
  constexpr int FIRST = OA::COPIES + OB::COPIES + (F8T ? 1 : 0), SECOND = OA::COPIES;
  __shared__ __align__(1024) char lds[2 * SLOT];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;

  TileOf w;
  if (!locate<T, WGRAD, BM, BN, BM / 2>(p, w)) return;
  const int wm = wave / WN, wn = (wave % WN) * WTN;
  // the tile's row of this lane in fragment i
  auto row_of = [&](int i) { return (i / SH) * (BM / 2) + wm * HALF + OA::row_of(i % SH, l16); };

  float4v acc[SM][SN] = {};
  const int steps = (w.k_end + OA::KS - 1) / OA::KS;
  if (steps > 0) {
    OA oa1, oa2;
    OB ob;
    oa1.init(w.A, p.lda, w.m0, w.m_end, w.k_end, wave, lane, wm * HALF);
    oa2.init(w.A, p.lda, w.m0 + BM / 2, w.m_end, w.k_end, wave, lane, wm * HALF);
    ob.init(w.B, p.ldb, w.n0, p.N, w.k_end, wave, lane, wn);
    const uint32_t lds0 =
        __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_char*)lds);
    OS os;
    if constexpr (F8T) os.init(p, w, steps, wave, lane);
    auto issue_first = [&](int kt) {
      const uint32_t at = lds0 + (uint32_t)((kt & 1) * SLOT);
      ob.issue(kt, at + B0, wave);
      oa1.issue(kt, at + A1, wave);
      if constexpr (F8T) os.issue(kt, at + S0);
    };
    auto issue_second = [&](int kt) {
      oa2.issue(kt, lds0 + (uint32_t)((kt & 1) * SLOT + A2), wave);
    };
    // Where k is contiguous, a row's last K step ends inside it and the rest came from beyond
    // the row: the last step's fragments are masked (a lane's 16-byte groups g and g + 4).
    int8v last_mask;
    if constexpr (AKC || BKC) {
      const int tail = (w.k_end - (steps - 1) * OA::KS) * T::BYTES;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int n = tail - 16 * (g + (x & 4)) - 4 * (x & 3);
        last_mask[x] = n >= 4 ? -1 : n <= 0 ? 0 : (int)((1u << (8 * n)) - 1u);
      }
    }

    int8v b[SN], a[2 * OA::READ];
    float s_a[SM];              // kFast8
    float4v s_b[SN];
    int x_a[SM], x_b[SN];       // kScaled8
    // fragments of A, READ of them at a time, into the two sets in turn
    auto read_a = [&](const char* slot, int i, bool masked) {
      const int at = (i / OA::READ & 1) * OA::READ;
      (i < SH ? oa1 : oa2).read(slot + (i < SH ? A1 : A2), i % SH, a + at);
      if (AKC && masked) a[at] &= last_mask;
    };
    auto set_of = [](int i) { return (i / OA::READ & 1) * OA::READ + i % OA::READ; };
    auto read_scales = [&](const char* slot) {
      if constexpr (F8T) {
        const char* table = slot + S0;
        if constexpr (HOW == kScaled8) {
#pragma unroll
          for (int i = 0; i < SM; ++i) x_a[i] = OS::a_byte(table, row_of(i));
#pragma unroll
          for (int j = 0; j < SN; ++j) x_b[j] = OS::b_byte(table, wn + OB::row_of(j, l16));
        } else {
#pragma unroll
          for (int i = 0; i < SM; ++i) s_a[i] = OS::a(table, row_of(i));
          if constexpr (HOW == kFast8Blocks) {
            const float block = OS::b(table, wn);
#pragma unroll
            for (int i = 0; i < SM; ++i) s_a[i] *= block;
          } else {
#pragma unroll
            for (int j = 0; j < SN; ++j) s_b[j] = OS::b4(table, wn + OB::row_of(j, 4 * g));
          }
        }
      }
    };
    // The sums of a step of 8-bit values are scaled and added kLag products behind, while the
    // matrix cores work on the next ones.
    constexpr int kLag = 2, kRing = 3;
    float4v d[kRing];
    auto product_of = [&](int s, const int8v& fa) {  // product s = i * SN + j of the step
      const int i = s / SN, j = s % SN;
      if constexpr (HOW == kScaled8) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], fa, acc[i][j], 0, 0, 0,
                                                                     x_b[j], 0, x_a[i]);
      } else if constexpr (F8T) {
        const float4v z = {0.0f, 0.0f, 0.0f, 0.0f};
        d[s % kRing] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            b[j], fa, z, 0, 0, 0, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      } else {
        acc[i][j] = mma_half<T>(half_of(b[j], 0), half_of(fa, 0), acc[i][j]);
        acc[i][j] = mma_half<T>(half_of(b[j], 1), half_of(fa, 1), acc[i][j]);
      }
    };
    auto product = [&](int s) { product_of(s, a[set_of(s / SN)]); };
    auto add = [&](int s) {
      if constexpr (F8T && HOW != kScaled8) {
        if (s < 0) return;
        const int i = s / SN, j = s % SN;
        const float4v v = d[s % kRing];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] += v[r] * (HOW == kFast8Blocks ? s_a[i] : s_a[i] * s_b[j][r]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    // Step kt, of which LEFT follow (2: two or more).  No branch inside: values that live across
    // branches cost registers that the wave does not have.
    auto step = [&](auto left, int kt) {
      constexpr int LEFT = decltype(left)::value;
      const char* slot = lds + (kt & 1) * SLOT;
      const char* next = lds + ((kt + 1) & 1) * SLOT;
      const uint32_t to = lds0 + (uint32_t)((kt & 1) * SLOT);
      int4v rb, ra, rs;  // sources of the copies for step kt + 2
      int done = 0;      // of them (a constant wherever it is used)
      if constexpr (LEFT == 0) {
        if constexpr (AKC) a[0] &= last_mask;
        if constexpr (BKC) {
#pragma unroll
          for (int j = 0; j < SN; ++j) b[j] &= last_mask;
        }
      }
#pragma unroll
      for (int i = 0; i < SM; ++i) {
        if (i == SH - 1) {
          part_barrier<LEFT == 0 ? 0 : FIRST + SECOND>();
          if constexpr (LEFT == 2) {
            rb = ob.words(kt + 2);
            ra = oa1.words(kt + 2);
            if constexpr (F8T) rs = os.words(kt + 2);
          }
        }
        if (i == SM - 1 && LEFT > 0) {
          part_barrier<LEFT == 2 ? SECOND + FIRST : SECOND>();
          if constexpr (LEFT == 2) ra = oa2.words(kt + 2);
          read_a(next, 0, false);
        }
        if (i + 1 < SM && (i + 1) % OA::READ == 0) read_a(slot, i + 1, LEFT == 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < SN; ++j) {
          product(i * SN + j);
          add(i * SN + j - kLag);
          // The copies go out between the products: a wave waits for each to be taken, 16
          // cycles a copy for all waves of the CU together.
          if constexpr (LEFT == 2) {
            if (i >= SH - 1 && i < SM - 1) {
              constexpr int SLOTS = SH * SN;
              const int at = (i - (SH - 1)) * SN + j;
              while (done * SLOTS < (at + 1) * FIRST) {
                if (done < OB::COPIES) ob.copy(done, rb, to + B0, wave);
                else if (done < OB::COPIES + OA::COPIES) oa1.copy(done - OB::COPIES, ra, to + A1, wave);
                else if constexpr (F8T) os.copy(rs, to + S0);
                ++done;
              }
            } else if (i == SM - 1 && j * OA::COPIES / SN != (j + 1) * OA::COPIES / SN) {
              oa2.copy(j * OA::COPIES / SN, ra, to + A2, wave);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          if (i == SM - 1 && LEFT > 0 && (j + 1) % OB::READ == 0)  // done with these columns
            ob.read(next + B0, j + 1 - OB::READ, b + j + 1 - OB::READ);
          if (i == SM - 1) __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int s = SM * SN - kLag; s < SM * SN; ++s) add(s);
      if constexpr (LEFT > 0) read_scales(next);
    };
    using Two = std::integral_constant<int, 2>;
    using One = std::integral_constant<int, 1>;
    using None = std::integral_constant<int, 0>;

    if (w.m_end - w.m0 <= BM / 2) {
      // Half a tile: the step's fragments go into registers at once, which frees the slot.
      issue_first(0);
      if (steps > 1) issue_first(1);
      int8v h[SH];
      for (int kt = 0; kt < steps; ++kt) {
        const char* slot = lds + (kt & 1) * SLOT;
        if (kt + 1 < steps) part_barrier<FIRST>();
        else part_barrier<0>();
#pragma unroll
        for (int j = 0; j < SN; j += OB::READ) ob.read(slot + B0, j, b + j);
#pragma unroll
        for (int i = 0; i < SH; i += OA::READ) oa1.read(slot + A1, i, h + i);
        read_scales(slot);
        part_barrier<63>();  // (the copies stay open)
        if (kt + 2 < steps) issue_first(kt + 2);
        if (kt + 1 == steps) {
          if constexpr (AKC) {
#pragma unroll
            for (int i = 0; i < SH; ++i) h[i] &= last_mask;
          }
          if constexpr (BKC) {
#pragma unroll
            for (int j = 0; j < SN; ++j) b[j] &= last_mask;
          }
        }
#pragma unroll
        for (int s = 0; s < SH * SN + kLag; ++s) {
          if (s < SH * SN) product_of(s, h[s / SN]);
          if (s >= kLag) add(s - kLag);
        }
      }
      store_tile<OB, F8T ? GEMM_LP_BF16 : T::CODE>(p, w, wn, g, acc, [&](int i) { return w.m0 + row_of(i); });
      return;
    }

    issue_first(0);
    issue_second(0);
    if (steps > 1) {
      issue_first(1);
      part_barrier<SECOND + FIRST>();
      issue_second(1);
    } else {
      part_barrier<0>();
    }
    read_a(lds, 0, false);
#pragma unroll
    for (int j = 0; j < SN; j += OB::READ) ob.read(lds + B0, j, b + j);
    read_scales(lds);
    for (int kt = 0; kt + 2 < steps; ++kt) step(Two{}, kt);
    if (steps > 1) step(One{}, steps - 2);
    step(None{}, steps - 1);
  }
  store_tile<OB, F8T ? GEMM_LP_BF16 : T::CODE>(p, w, wn, g, acc, [&](int i) { return w.m0 + row_of(i); });
}

}  // namespace gemmlp
