// The units that the pipelined product kernels are compiled in: an element type and the order
// of the operands (does k, the contraction, lie contiguous in A and in B).
#pragma once

#include "lp_common.h"

namespace gemmlp {

// Tiles of the pipelined kernels (K4: four groups of waves share the K steps).
enum { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTile64K4 = 3, kTileCount = 4 };
struct TileSize {
  int bm, bn, threads;
};
constexpr TileSize kTiles[] = {{256, 256, 512}, {128, 128, 256}, {64, 64, 256}, {64, 64, 1024}};

template <class T, bool A, bool B, bool W, int H>
struct Unit {
  using type = T;
  static constexpr bool AKC = A, BKC = B, WGRAD = W;
  static constexpr int HOW = H;
};
template <int UNIT>
struct UnitOf;
// 16- and 32-bit: X W^T, X W, and the weight gradient
template <> struct UnitOf<0> : Unit<Bf16, true, true, false, 0> {};
template <> struct UnitOf<1> : Unit<Bf16, true, false, false, 0> {};
template <> struct UnitOf<2> : Unit<Bf16, false, false, true, 0> {};
template <> struct UnitOf<3> : Unit<F16, true, true, false, 0> {};
template <> struct UnitOf<4> : Unit<F16, true, false, false, 0> {};
template <> struct UnitOf<5> : Unit<F16, false, false, true, 0> {};
template <> struct UnitOf<6> : Unit<F32, true, true, false, 0> {};
template <> struct UnitOf<7> : Unit<F32, true, false, false, 0> {};
template <> struct UnitOf<8> : Unit<F32, false, false, true, 0> {};
// 8-bit (the last number is lp_pipe.h's HOW): B's scales by columns, by blocks, and exponents for
// scales
template <> struct UnitOf<9> : Unit<F8, true, true, false, 0> {};
template <> struct UnitOf<10> : Unit<F8, true, true, false, 1> {};
template <> struct UnitOf<11> : Unit<F8, true, true, false, 2> {};
constexpr int kUnits = 12;

// The kernel of a tile, or NULL where the unit has none; staged: for operands of any alignment.
LpKernel pipe_kernel_0(int tile, bool staged);
LpKernel pipe_kernel_1(int tile, bool staged);
LpKernel pipe_kernel_2(int tile, bool staged);
LpKernel pipe_kernel_3(int tile, bool staged);
LpKernel pipe_kernel_4(int tile, bool staged);
LpKernel pipe_kernel_5(int tile, bool staged);
LpKernel pipe_kernel_6(int tile, bool staged);
LpKernel pipe_kernel_7(int tile, bool staged);
LpKernel pipe_kernel_8(int tile, bool staged);
LpKernel pipe_kernel_9(int tile, bool staged);
LpKernel pipe_kernel_10(int tile, bool staged);
LpKernel pipe_kernel_11(int tile, bool staged);

}  // namespace gemmlp
