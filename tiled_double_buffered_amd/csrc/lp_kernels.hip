// The pipelined product kernels of one element type and operand order, compiled once for each
// (LP_UNIT) so that they build in parallel.
#include <hip/hip_runtime.h>

#include "lp_deep.h"
#include "lp_pipe.h"
#include "lp_units.h"

#ifndef LP_UNIT
#error "compile with -DLP_UNIT=<number>"
#endif

namespace gemmlp {

template <class U, int BM, int BN, int WM, int WN, bool STAGED, int KG = 1>
constexpr LpKernel pipe() {
  return &lp_pipe_kernel<typename U::type, U::AKC, U::BKC, U::WGRAD, BM, BN, WM, WN, U::HOW,
                         STAGED, KG>;
}

template <class U>
static LpKernel pick(int tile, bool staged) {
  using T = typename U::type;
  if (tile == kTile256 && !staged) {
    // 8-bit values, converted on the way, need more registers than a wave of this kernel has
    if constexpr (T::BYTES != 1) return &lp_deep_kernel<T, U::AKC, U::BKC, U::WGRAD>;
  }
  if (tile == kTile128) {
    // (these need a few registers more than two workgroups of a CU have)
    if constexpr (T::BYTES == 1 && U::HOW == kScaleRows)
      if (staged) return nullptr;
    return staged ? pipe<U, 128, 128, 2, 2, !(T::BYTES == 1 && U::HOW == kScaleRows)>()
                  : pipe<U, 128, 128, 2, 2, false>();
  }
  if (tile == kTile64)
    return staged ? pipe<U, 64, 64, 2, 2, true>() : pipe<U, 64, 64, 2, 2, false>();
  if (tile == kTile64K4)
    return staged ? pipe<U, 64, 64, 2, 2, true, 4>() : pipe<U, 64, 64, 2, 2, false, 4>();
  return nullptr;
}

#define LP_CAT2(a, b) a##b
#define LP_CAT(a, b) LP_CAT2(a, b)
LpKernel LP_CAT(pipe_kernel_, LP_UNIT)(int tile, bool staged) {
  return pick<UnitOf<LP_UNIT>>(tile, staged);
}

}  // namespace gemmlp
