// The pipelined product kernels of one element type and operand order, compiled once for each
// (LP_UNIT) so that they build in parallel.
#include <hip/hip_runtime.h>

#include "lp_pipe.h"
#include "lp_units.h"

#ifndef LP_UNIT
#error "compile with -DLP_UNIT=<number>"
#endif

namespace gemmlp {

template <int UNIT>
static LpKernel pick(int tile) {
  using U = UnitOf<UNIT>;
  using T = typename U::type;
  // (8-bit values through the 16-bit instruction need more registers than a wave of the
  // large tile has)
  constexpr bool kLarge = U::FAST8 || T::BYTES != 1;
  if constexpr (kLarge)
    if (tile == kTile256) return &lp_pipe_kernel<T, U::AKC, U::BKC, U::WGRAD, 256, 256, 2, 4, U::FAST8>;
  if (tile == kTile128) return &lp_pipe_kernel<T, U::AKC, U::BKC, U::WGRAD, 128, 128, 2, 2, U::FAST8>;
  return nullptr;
}

#define LP_CAT2(a, b) a##b
#define LP_CAT(a, b) LP_CAT2(a, b)
LpKernel LP_CAT(pipe_kernel_, LP_UNIT)(int tile) { return pick<LP_UNIT>(tile); }

}  // namespace gemmlp
