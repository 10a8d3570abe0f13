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

template <int UNIT>
static LpKernel pick(int tile) {
  using U = UnitOf<UNIT>;
  using T = typename U::type;
  if (tile == kTile256) {
    // 8-bit values through the 16-bit instruction, or with a scale for each column, need more
    // registers than a wave of the deep kernel has
    if constexpr (T::BYTES != 1 || U::HOW == kFast8Blocks)
      return &lp_deep_kernel<T, U::AKC, U::BKC, U::WGRAD, U::HOW>;
    else if constexpr (U::HOW == kFast8Rows)
      return &lp_pipe_kernel<T, U::AKC, U::BKC, U::WGRAD, 256, 256, 2, 4, U::HOW>;
  }
  if (tile == kTile128) return &lp_pipe_kernel<T, U::AKC, U::BKC, U::WGRAD, 128, 128, 2, 2, U::HOW>;
  if (tile == kTile64) return &lp_pipe_kernel<T, U::AKC, U::BKC, U::WGRAD, 64, 64, 2, 2, U::HOW>;
  return nullptr;
}

#define LP_CAT2(a, b) a##b
#define LP_CAT(a, b) LP_CAT2(a, b)
LpKernel LP_CAT(pipe_kernel_, LP_UNIT)(int tile) { return pick<LP_UNIT>(tile); }

}  // namespace gemmlp
