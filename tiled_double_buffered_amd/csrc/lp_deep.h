// The pipelined product kernel for large products of 16- and 32-bit values: 256 x 256 tiles, eight
// waves of 128 x 64, two LDS slots refilled in halves, so that a copy has one and a half K steps
// to land.
//
// The kernel of lp_pipe.h starts a step's copies when the slot's last reader is done and needs
// them one step later, and waits for them.  Here each slot has three parts that are freed at
// different times: B, which a wave holds in registers for the whole step, the upper half A1 of
// A's rows, which the step's first products read, and the lower half A2.  A step has two
// barriers:
//   middle (before the products of the last A1 fragment): B, A1 of this step are read by all
//     waves, A2 of this step has landed; the copies of B, A1 two steps on start;
//   end (before the products of the last two A2 fragments): A2 of this step is read, B and A1
//     of the next have landed; the copies of A2 two steps on start.  The last two rows of
//     products go column by column, so that B's fragments are replaced one by one.
// A tile of 128 rows or fewer leaves A2 and its products out.
// Copies complete in order, so a wave waits until no more are open than were started after the
// part it needs.
//
// Measured on MI355X at 8192^3, warm: bf16 X W^T 763 us, X W 766, weight gradient 745 (1.4 to
// 1.5 PFLOP/s, the matrix cores busy 74 to 75 % of the time at the 1.8 GHz that the power limit
// leaves); FP32 137 to 148 TFLOP/s.  A step's copies, reads and barriers take about as long as its
// products: the spread copies, B replaced piece by piece and scalar walks are what overlaps them.
// Three half slots for half tiles, wave priorities, and workgroups that stay and fetch their next
// tile's first steps before they store made no difference.  Four waves of 128 x 128 read a third
// less from LDS, which is faster while the power limit holds (bf16 8192^3: 751 us, where eight
// took 788) but slower for ragged groups (16384 rows of 32 experts, X W 318 us against 311,
// X W^T 336 against 323), whose half tiles then lack waves to hide their waits.
#pragma once

#include <type_traits>

#include "lp_pipe.h"

namespace gemmlp {

template <class T, bool AKC, bool BKC, bool WGRAD>
__global__ __launch_bounds__(512) void lp_deep_kernel(LpArgs p) {
  constexpr int BM = 256, BN = 256, WN = 4, WAVES = 8;
  constexpr int WTM = 128, WTN = 64, HALF = WTM / 2, SM = 8, SN = 4, SH = SM / 2;
  static_assert(T::BYTES != 1, "not enough registers");
  constexpr bool PACK = T::BYTES == 2;
  using OA = PipeOperand<T, AKC, BM / 2, HALF, WAVES>;
  using OB = PipeOperand<T, BKC, BN, WTN, WAVES, PACK>;
  constexpr int A1 = 0, A2 = OA::BYTES, B0 = 2 * OA::BYTES, SLOT = B0 + OB::BYTES;
  constexpr int FIRST = OA::COPIES + OB::COPIES, SECOND = OA::COPIES;
  __shared__ __align__(1024) char lds[2 * SLOT];
  static_assert(sizeof(lds) <= 160 * 1024, "LDS of one CU");
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
    // (each is called for one step after another)
    Walk to_b, to_a1, to_a2;
    ob.start(to_b);
    oa1.start(to_a1);
    oa2.start(to_a2);
    auto issue_first = [&](int kt) {
      const uint32_t at = lds0 + (uint32_t)((kt & 1) * SLOT);
      const int4v rb = to_b.next(), ra = to_a1.next();
#pragma unroll
      for (int i = 0; i < OB::COPIES; ++i) ob.copy(i, rb, at + B0, wave);
#pragma unroll
      for (int i = 0; i < OA::COPIES; ++i) oa1.copy(i, ra, at + A1, wave);
    };
    auto issue_second = [&](int kt) {
      const uint32_t at = lds0 + (uint32_t)((kt & 1) * SLOT);
      const int4v ra = to_a2.next();
#pragma unroll
      for (int i = 0; i < OA::COPIES; ++i) oa2.copy(i, ra, at + A2, wave);
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

    int8v b[SN], a[OA::READ == 1 ? 4 : 2 * OA::READ];
    // Fragment i of A is held in a[set_of(i)] from before its products to their end; the first
    // of a step is read while the last two of the step before are still in use.
    auto set_of = [](int i) { return OA::READ > 1 ? i : i == 0 ? 2 : i == SM - 1 ? 3 : 1 - (i & 1); };
    static_assert(OA::READ == 1 || 2 * OA::READ == SM, "two groups of fragments");
    auto read_a = [&](const char* slot, int i, bool masked) {
      (i < SH ? oa1 : oa2).read(slot + (i < SH ? A1 : A2), i % SH, a + set_of(i));
      if (AKC && masked) a[set_of(i)] &= last_mask;
    };
    // Product number s of a step: row by row, the last two rows column by column.
    constexpr int ROWS = SM - 2;
    auto row_at = [](int s) { return s < ROWS * SN ? s / SN : ROWS + (s & 1); };
    auto col_at = [](int s) { return s < ROWS * SN ? s % SN : (s - ROWS * SN) / 2; };
    auto product_of = [&](int i, int j, const int8v& fa) {
      acc[i][j] = mma_half<T>(half_of(b[j], 0), half_of(fa, 0), acc[i][j]);
      acc[i][j] = mma_half<T>(half_of(b[j], 1), half_of(fa, 1), acc[i][j]);
    };
    // Step kt, of which LEFT follow (2: two or more).  No branch inside: values that live across
    // branches cost registers that the wave does not have.
    auto step = [&](auto left, int kt) {
      constexpr int LEFT = decltype(left)::value;
      const char* slot = lds + (kt & 1) * SLOT;
      const char* next = lds + ((kt + 1) & 1) * SLOT;
      const uint32_t to = lds0 + (uint32_t)((kt & 1) * SLOT);
      int4v rb, ra;  // sources of the copies for step kt + 2
      int done = 0;  // of them (a constant wherever it is used)
      if constexpr (LEFT == 0) {
        if constexpr (AKC) a[set_of(0)] &= last_mask;
        if constexpr (BKC) {
#pragma unroll
          for (int j = 0; j < SN; ++j) b[j] &= last_mask;
        }
      }
#pragma unroll
      for (int s = 0; s < SM * SN; ++s) {
        const int i = row_at(s), j = col_at(s);
        if (s == (SH - 1) * SN) {
          part_barrier<LEFT == 0 ? 0 : FIRST + SECOND>();
          if constexpr (LEFT == 2) {
            rb = to_b.next();
            ra = to_a1.next();
          }
        }
        if (s == ROWS * SN && LEFT > 0) {
          part_barrier<LEFT == 2 ? SECOND + FIRST : SECOND>();
          if constexpr (LEFT == 2) ra = to_a2.next();
          read_a(next, 0, false);
        }
        if (j == 0 && i < ROWS && (i + 1) % OA::READ == 0) read_a(slot, i + 1, LEFT == 0);
        if (OA::READ == 1 && s == SH * SN + 1)  // well before the end barrier
          read_a(slot, SM - 1, LEFT == 0);
        __builtin_amdgcn_sched_barrier(0);
        product_of(i, j, a[set_of(i)]);
        // The copies go out between the products: a wave waits for each to be taken, 16 cycles
        // a copy for all waves of the CU together.
        if constexpr (LEFT == 2) {
          if (s >= (SH - 1) * SN && s < ROWS * SN) {
            constexpr int SLOTS = (ROWS - SH + 1) * SN;
            while (done * SLOTS < (s - (SH - 1) * SN + 1) * FIRST) {
              if (done < OB::COPIES) ob.copy(done, rb, to + B0, wave);
              else oa1.copy(done - OB::COPIES, ra, to + A1, wave);
              ++done;
            }
          } else if (s >= ROWS * SN) {
            constexpr int SLOTS = 2 * SN;
            const int n = s - ROWS * SN;
            if (n * OA::COPIES / SLOTS != (n + 1) * OA::COPIES / SLOTS)
              oa2.copy(n * OA::COPIES / SLOTS, ra, to + A2, wave);
          }
        }
        if (LEFT > 0 && s >= ROWS * SN && row_at(s) == SM - 1 && (j + 1) % OB::READ == 0)
          ob.read(next + B0, j + 1 - OB::READ, b + j + 1 - OB::READ);  // done with these columns
        __builtin_amdgcn_sched_barrier(0);
      }
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
        for (int s = 0; s < SH * SN; ++s) product_of(s / SN, s % SN, h[s / SN]);
      }
      store_tile<OB, T::CODE>(p, w, wn, g, acc, [&](int i) { return w.m0 + row_of(i); });
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
    for (int kt = 0; kt + 2 < steps; ++kt) step(Two{}, kt);
    if (steps > 1) step(One{}, steps - 2);
    step(None{}, steps - 1);
  }
  store_tile<OB, T::CODE>(p, w, wn, g, acc, [&](int i) { return w.m0 + row_of(i); });
}

}  // namespace gemmlp
